// kv_attn.cuh -- attention of new tokens over the paged cache, of 16 or of
// 4 bits, and the merge of units that were cut between CTAs.
//
// A unit is one token row and the G query heads (at most 8 kNt) that share a
// kv head: all of them have the same keys, so nothing is masked per query,
// and a key that is not in the set is never loaded (its slot counts as
// zeros), whatever the cache holds there.
//
// kPack: a unit is a tile of consecutive rows of a sequence (drafts, prompts),
// whose windows differ at the ends.  The keys that all rows see are taken as
// above; of the others each score is masked by its row's window, and a value
// that is no number (infinity, NaN) is kept from the rows that do not see it: 0
// times it is not 0, so then the products are taken row by row, with the row's
// own keys alone.  (Such a step costs a few times as much; it is rare.)
//
// Bound: the cache's bytes.  A key's row is read once for at most 16 query
// heads, so the intensity is at most 16 flops a byte in 16 bits (measured: 16
// sequences of 16384 to 32768 tokens, 8 kv heads of 128, bf16: 1.63 GB in 244
// us, the rate of a plain copy; 16 sequences of 4 drafted tokens, 4000 keys, 32
// heads on 8 of 128: 262 MB in 53 us).  Both products are written transposed,
// S^T = K Q^T and O^T = V^T P^T (m16n8k16 with 16 keys, or 16 value dimensions,
// as M and 8 query heads as N), which needs half the MMAs and accumulators of
// the other order when there are few heads.
//   lane (g, c) = (lane / 4, lane % 4).  K: the lane reads the 16-byte chunks
//   c, c + 4, .. of keys g and g + 8; the MMA's k index is a permutation of
//   the head dimension, the same for Q.  V: chunk g (and g + 8) of keys 2c,
//   2c + 1, 2c + 8, 2c + 9, whose halves are paired by byte permutes.  P^T
//   goes from accumulator to operand layout by one matrix transpose
//   (movmatrix) per 8 keys.
// A CTA's four warps take 16 or 32 keys each of a 64- or 128-key block; a warp
// keeps its own running maximum, sum and O, joined through shared memory when
// the unit's piece ends.  Each warp has a ring of stages in shared memory that
// it fills itself with cp.async, one block ahead of the one it computes (two
// ahead measured 4 % slower over long sequences), across unit boundaries too
// (short windows are a few blocks long); the page table is read one block before
// that, and the next unit's queries while the last block of a unit is computed.
//
// 4 bits: a group of 32 values is mid + scale (c - 8).  A code or'ed into the
// mantissa of 1024 is an f16 (1024 + c, or 1024 + 16 c for a nibble four bits
// up), so all MMAs are f16 here.  K stays codes: q . k = sum over groups of
// scale (sum of q (c - 8)) + mid (sum of q) in fp32, the 1024 taken off the
// fp32 sum (what that loses is 1024 steps of 2^-24 of the q sum).  Queries are
// brought to +-2^14 by a power of two for it, and every second one, whose codes
// are 16 times theirs, to 2^10: f16 holds them exactly down to 2^-23 of the
// largest, and to 2^-34 of it below.  V is made f16 values, one
// rounding (2^-11); those past its range are halved first and weigh twice
// (double_large).  Bound here: instructions, about 28 a key and warp at d =
// 128, half of them integer ones to spread nibbles (4 sequences of 32768 to
// 65536 tokens, 8 kv heads of 128: 264 MB in 79 us, 51 % of the copy rate).
//
// Rounding: scores, maxima, sums and O in fp32.  P goes to the tensor cores in
// two bf16 (2^-15) or f16 parts (2^-20): the second part's MMAs are free where
// the bytes bound it.  Over 4 bits, where V is rounded to f16 anyway, P is one
// f16 (2^-11) with bf16 queries and two with f16 ones.
#pragma once
#include "kv_plan.cuh"
#include "lf_common.cuh"
#include "ptx.cuh"

namespace lf {

constexpr int kKvWarps = 4;
constexpr int kKvThreads = kKvWarps * 32;
constexpr int kStages = 2;

// Steps of 16 keys that a warp takes at once: two over 4 bits, so that what a
// step costs besides its keys (the walk, the vote on the base) is paid half as
// often (102 -> 88 us at 1.6 M keys of d = 128); one over 16 bits, where 32
// rows a stage would leave an SM half the warps (d = 64, batch of short
// windows: 7.4 against 9.1 us).
__host__ __device__ constexpr int kv_sub(int bits) { return bits == 16 ? 1 : 2; }
__host__ __device__ constexpr int kv_block(int bits) { return kKvWarps * 16 * kv_sub(bits); }

// Query rows of a tile, at most.  Over 4 bits of d = 128 16 rows spill (16
// sequences of 6 drafts, 4000 keys, 32 heads on 8: 109 us against 88 with 8).
// Of d = 64 they spill too (56 bytes a thread, 164 with f16 queries) but take
// less on prompts: 4096 rows, 12 heads, window 256, 84 us against 105 with 8 (f16
// 104 : 109); the drafts above 43.5 : 46.3 (f16 56.0 : 48.5).
__host__ __device__ constexpr int kv_tile_rows(int d, int bits) { return d == 128 && bits == 4 ? 8 : 16; }

// CTAs of four warps that an SM holds at once, by registers (128 to 255 a
// thread).
__host__ __device__ constexpr int kv_ctas_per_sm(int d, int bits, bool two, bool pack) {
    return pack ? (d == 128 ? 2 : 3) : d == 64 ? (two || bits == 4 ? 3 : 4) : (bits == 16 || two ? 2 : 3);
}

// A stage: for each 16 keys the K rows, the V rows, and for 4 bits their parameters.
template <int HD, int kBits>
struct KvStage {
    static constexpr int kSub = kv_sub(kBits);
    static constexpr int kRow = kBits == 16 ? HD * 2 : HD / 2;
    static constexpr int kPar = kBits == 16 ? 0 : HD / 8;
    static constexpr int kV = 16 * kRow, kKp = 32 * kRow, kVp = kKp + 16 * kPar;
    static constexpr int kSubBytes = kVp + 16 * kPar;
    static constexpr int kBytes = kSub * kSubBytes;
};

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
    float* part;         // [2 G][unit_rows][d + 4]
    int N, n_pages, log_page, max_pages;
    int kv_heads, group, nsub, gs, r, n_global, G;
    int o_wide;          // output rows begin at 8-byte boundaries
    int unit_rows;       // most query rows of a unit: gs times the rows of a tile
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

// The same with C = 0.
template <bool kHalf>
__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
    if constexpr (kHalf)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t pack_f16x2_rz(float lo, float hi) {  // toward 0
    uint32_t y;
    asm("cvt.rz.f16x2.f32 %0, %2, %1;" : "=r"(y) : "f"(lo), "f"(hi));
    return y;
}

__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Two nibbles of x, bits 0-3 and 16-19 (kUp: 4-7 and 20-23), as f16 1024 + c (1024 + 16 c).
template <bool kUp>
__device__ __forceinline__ uint32_t code_pair(uint32_t x) {
    return (x & (kUp ? 0x00f000f0u : 0x000f000fu)) | 0x64006400u;
}
// ... and as c - 8, exactly.
template <bool kUp>
__device__ __forceinline__ __half2 code_value(uint32_t x) {
    const uint32_t y = code_pair<kUp>(x), bias = kUp ? 0xd480d480u : 0xe408e408u;  // -72, -1032
    const __half2 b = *reinterpret_cast<const __half2*>(&bias), v = *reinterpret_cast<const __half2*>(&y);
    if constexpr (kUp) return __hfma2(v, __float2half2_rn(0.0625f), b);
    else return __hadd2(v, b);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {  // zeros if not there
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(there ? 8 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// 16-bit rows: 16-byte chunk x of row r is at chunk x ^ swz(r), so that the K
// reads (rows g, chunks c of 8 lanes: two rows, four chunks) and the V reads
// (rows 2c, chunks g: four rows, two chunks) both meet all 32 banks once.
__device__ __forceinline__ int swz(int r) { return (((r ^ (r >> 2)) & 1) << 2) | (r & 2); }
// 4-bit V rows: key k's place, so that keys 2c (2c + 1, ..) are beside each other.
__device__ __forceinline__ int v_place(int k) { return (k & 8) | ((k & 1) << 2) | ((k >> 1) & 3); }

// Starts the copies of a warp's keys into a stage; lane i has key i's row of
// the cache, -1: none (zeros).
template <int HD, int kBits>
__device__ __forceinline__ void kv_issue(const KvAttnParams& p, uint32_t stage, int row, int lane) {
    using St = KvStage<HD, kBits>;
    if constexpr (kBits == 16) {
        constexpr int kChunks = St::kRow / 16;  // per row: 8 or 16; 32 lanes take 32 / kChunks whole rows at a time
        const int x = lane % kChunks;
#pragma unroll
        for (int i = 0; i < kChunks / 2; ++i) {
            const int r = (i * 32 + lane) / kChunks, at = __shfl_sync(~0u, row, r);
            const int64_t off = int64_t(max(at, 0)) * St::kRow + 16 * x;
            const uint32_t dst = stage + r * St::kRow + 16 * (x ^ swz(r));
            cp_async16(dst, p.k + off, at >= 0);
            cp_async16(dst + St::kV, p.v + off, at >= 0);
        }
    } else {
        // two lanes a row, 32 bytes of it at a time: an address serves a whole row
        const int x = 16 * (lane & 1), k = lane >> 1;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int at = __shfl_sync(~0u, row, 16 * u + k);
            const int64_t off = int64_t(max(at, 0)) * St::kRow + x;
            const uint8_t *ks = p.k + off, *vs = p.v + off;
            const uint32_t dk = stage + u * St::kSubBytes + k * St::kRow + x;
            const uint32_t dv = stage + u * St::kSubBytes + St::kV + v_place(k) * St::kRow + x;
#pragma unroll
            for (int j = 0; j < St::kRow; j += 32) {
                cp_async16(dk + j, ks + j, at >= 0);
                cp_async16(dv + j, vs + j, at >= 0);
            }
        }
        // lane i: the parameters of key i
        const int64_t off = int64_t(max(row, 0)) * St::kPar;
        const uint32_t dst = stage + (lane >> 4) * St::kSubBytes + (lane & 15) * St::kPar;
        if constexpr (St::kPar == 16) {
            cp_async16(dst + St::kKp, p.k_par + off, row >= 0);
            cp_async16(dst + St::kVp, p.v_par + off, row >= 0);
        } else {
            cp_async8(dst + St::kKp, p.k_par + off, row >= 0);
            cp_async8(dst + St::kVp, p.v_par + off, row >= 0);
        }
    }
}

// What a lane takes of a stage.
template <int HD, int kBits>
struct KvRegs;
template <int HD>
struct KvRegs<HD, 16> {
    uint4 k[2][HD / 32];  // keys g, g + 8: chunks c, c + 4, ..
    uint4 v[4][HD / 64];  // keys 2c, 2c + 1, 2c + 8, 2c + 9: chunks g, g + 8
    __device__ __forceinline__ void load_k(const uint8_t* s, int g, int c) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < HD / 32; ++j)
                k[i][j] = *reinterpret_cast<const uint4*>(s + (g + 8 * i) * (HD * 2) + 16 * ((c + 4 * j) ^ swz(g + 8 * i)));
    }
    __device__ __forceinline__ void load_v(const uint8_t* s, int g, int c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 2 * c + (i & 1) + 8 * (i >> 1);
#pragma unroll
            for (int j = 0; j < HD / 64; ++j)
                v[i][j] = *reinterpret_cast<const uint4*>(s + KvStage<HD, 16>::kV + r * (HD * 2) + 16 * ((g + 8 * j) ^ swz(r)));
        }
    }
};
template <int W>
__device__ __forceinline__ void load_words(uint32_t (&x)[W], const uint8_t* at) {
    static_assert(W == 1 || W == 2 || W == 4, "");
    if constexpr (W == 1) {
        x[0] = *reinterpret_cast<const uint32_t*>(at);
    } else if constexpr (W == 2) {
        const uint2 t = *reinterpret_cast<const uint2*>(at);
        x[0] = t.x; x[1] = t.y;
    } else {
        const uint4 t = *reinterpret_cast<const uint4*>(at);
        x[0] = t.x; x[1] = t.y; x[2] = t.z; x[3] = t.w;
    }
}
template <int HD>
struct KvRegs<HD, 4> {
    static constexpr int kGroups = HD / 32;
    using St = KvStage<HD, 4>;
    uint32_t k[2][kGroups];   // keys g, g + 8: word [c] of each group
    uint32_t v[4][HD / 64];   // keys 2c, ..: units [g] of two groups each
    uint32_t kp[2][kGroups];  // keys g, g + 8: (scale, mid) of each group
    uint32_t vp[4][kGroups];  // keys 2c, ..
    __device__ __forceinline__ void load_k(const uint8_t* s, int g, int c) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            load_words(k[i], s + (g + 8 * i) * St::kRow + c * (4 * kGroups));
            load_words(kp[i], s + St::kKp + (g + 8 * i) * St::kPar);
        }
    }
    __device__ __forceinline__ void load_v(const uint8_t* s, int g, int c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = 2 * c + (i & 1) + 8 * (i >> 1);
            load_words(v[i], s + St::kV + v_place(k) * St::kRow + g * (2 * kGroups));
            load_words(vp[i], s + St::kVp + k * St::kPar);
        }
    }
};

__device__ __forceinline__ float2 par_of(uint32_t x) {  // (scale, mid)
    return __half22float2(*reinterpret_cast<const __half2*>(&x));
}

// The warp's state of a unit.  Query heads 8 n + 2c and 8 n + 2c + 1 of this
// lane are columns 0 and 1 of its n-th tile.
template <int HD, int kBits, bool kHalf, int kNt, bool kPack>
struct KvState {
    static constexpr int kGroups = HD / 32;
    static constexpr bool kSplitP = kBits == 4 && kHalf;
    // P = 2^(score - base + kLift), at most 2^(kLift + kRoom).  An f16 P is lifted so that a weight 2^-36 of the
    // largest still counts (2^-37 over 16 bits): a million such keys are 2^-16 of the sum.  Over 4 bits one power of two is
    // left free for double_large; over 16 bits it goes into the lift, since no weight is under 2^-23 (values()).
    static constexpr float kLift = kBits == 4 ? 11.f : kHalf ? 12.f : 0.f, kRoom = kBits == 4 || kHalf ? 3.f : 8.f;
    uint32_t q[kNt][HD / 16][2];
    float o[kNt][HD / 16][4];
    float m[kNt][2], l[kNt][2];  // (o[.][4 j + t][i]: dimension 64 j + 8 g + 2 t + (i >> 1); 4 bits: [2 j + t]: 32 j + 4 g + ..)
    // 4 bits: sums of the scaled q over a group, minus what the codes' 1024 + 8 adds to its products, and the scale of
    // scores (16 bits: the caller's)
    float qs[kBits == 4 ? kNt : 1][kBits == 4 ? kGroups : 1][2], qa[kBits == 4 ? kNt : 1][kBits == 4 ? kGroups : 1][2];
    float rs[kNt][2];

    // Where query row i of a unit is from its first one on, in elements.
    static __device__ __forceinline__ int64_t row_at(int i, int gs, int64_t token, int64_t head) {
        if constexpr (kPack) return (i / gs) * token + (i % gs) * head;
        else return i * head;
    }

    // The unit's queries as they are in memory: lane (g, c) takes chunks c, c + 4, .. of query row 8 n + g (heads of a
    // token, then of the next).
    static __device__ __forceinline__ void load_q(uint4 (&x)[kNt][HD / 32], const KvAttnParams& p, const uint8_t* qrow,
                                                  int rows, int lane) {
        const int g = lane >> 2, c = lane & 3;
#pragma unroll
        for (int n = 0; n < kNt; ++n)
#pragma unroll
            for (int j = 0; j < HD / 32; ++j)
                x[n][j] = 8 * n + g < rows
                              ? __ldg(reinterpret_cast<const uint4*>(qrow + 2 * row_at(8 * n + g, p.gs, p.q_row, p.q_head)) +
                                      c + 4 * j)
                              : make_uint4(0, 0, 0, 0);
    }

    __device__ __forceinline__ void begin(const uint4 (&x)[kNt][HD / 32], int lane, float sl2) {
        const int c = lane & 3;
#pragma unroll
        for (int n = 0; n < kNt; ++n) {
            if constexpr (kBits == 16) {
#pragma unroll
                for (int j = 0; j < HD / 32; ++j) {
                    q[n][2 * j][0] = x[n][j].x; q[n][2 * j][1] = x[n][j].y;
                    q[n][2 * j + 1][0] = x[n][j].z; q[n][2 * j + 1][1] = x[n][j].w;
                }
                rs[n][0] = rs[n][1] = sl2;
            } else {
                // query head g of the tile: its largest |q|, and the power of two that brings it to [2^13, 2^14)
                float f[HD / 32][8], top = 0.f;
#pragma unroll
                for (int j = 0; j < HD / 32; ++j) {
                    const uint32_t w[4] = {x[n][j].x, x[n][j].y, x[n][j].z, x[n][j].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float2 v;
                        if constexpr (kHalf) v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                        else v = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
                        f[j][2 * i] = v.x;
                        f[j][2 * i + 1] = v.y;
                        top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
                    }
                }
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
                const uint32_t e = max(__float_as_uint(top) >> 23, 14u);  // 255: an infinity: no scaling; under 2^-113: as that
                const float down = e == 255 ? 1.f : __uint_as_float((267u - e) << 23);
                const float up = e == 255 ? 1.f : __uint_as_float((e - 13u) << 23);
                rs[n][0] = sl2 * __shfl_sync(~0u, up, 8 * c);
                rs[n][1] = sl2 * __shfl_sync(~0u, up, 8 * c + 4);
#pragma unroll
                for (int j = 0; j < HD / 32; ++j) {
                    // values (i, i + 4) of the chunk beside each other, as the codes of a word; the odd ones' codes are
                    // 16 times theirs
                    float even = 0.f, odd = 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float by = (i & 1) ? down * 0.0625f : down;
                        const __half2 h = __floats2half2_rn(f[j][i] * by, f[j][i + 4] * by);
                        q[n][2 * j + (i >> 1)][i & 1] = *reinterpret_cast<const uint32_t*>(&h);
                        const float2 v = __half22float2(h);
                        if (i & 1) odd += v.x + v.y;
                        else even += v.x + v.y;
                    }
                    float sum = fmaf(16.f, odd, even), base = -fmaf(1024.f, even + odd, 8.f * sum);
                    sum += __shfl_xor_sync(~0u, sum, 1);
                    base += __shfl_xor_sync(~0u, base, 1);
                    sum += __shfl_xor_sync(~0u, sum, 2);
                    base += __shfl_xor_sync(~0u, base, 2);
                    qs[n][j][0] = __shfl_sync(~0u, sum, 8 * c);
                    qs[n][j][1] = __shfl_sync(~0u, sum, 8 * c + 4);
                    qa[n][j][0] = __shfl_sync(~0u, base, 8 * c);
                    qa[n][j][1] = __shfl_sync(~0u, base, 8 * c + 4);
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

    // The scores of 16 keys: s[n][i] of key g (i < 2) or g + 8 and query head 8 n + 2c + (i & 1).
    __device__ __forceinline__ void scores(float (&s)[kNt][4], const uint8_t* sub, int g, int c) {
        KvRegs<HD, kBits> x;
        x.load_k(sub, g, c);
        if constexpr (kBits == 16) {
#pragma unroll
            for (int j = 0; j < HD / 32; ++j)
#pragma unroll
                for (int n = 0; n < kNt; ++n) {
                    if (j == 0)
                        mma16816_first<kHalf>(s[n], x.k[0][j].x, x.k[1][j].x, x.k[0][j].y, x.k[1][j].y, q[n][0][0],
                                              q[n][0][1]);
                    else
                        mma16816<kHalf>(s[n], x.k[0][j].x, x.k[1][j].x, x.k[0][j].y, x.k[1][j].y, q[n][2 * j][0],
                                        q[n][2 * j][1]);
                    mma16816<kHalf>(s[n], x.k[0][j].z, x.k[1][j].z, x.k[0][j].w, x.k[1][j].w, q[n][2 * j + 1][0],
                                    q[n][2 * j + 1][1]);
                }
        } else {
            float2 sum[kNt][2];
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
                uint32_t a[2][4];
                float2 scale[2], mid[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t w = x.k[i][j], w8 = w >> 8;
                    a[i][0] = code_pair<false>(w);
                    a[i][1] = code_pair<true>(w);
                    a[i][2] = code_pair<false>(w8);
                    a[i][3] = code_pair<true>(w8);
                    const float2 f = par_of(x.kp[i][j]);
                    scale[i] = make_float2(f.x, f.x);
                    mid[i] = make_float2(f.y, f.y);
                }
#pragma unroll
                for (int n = 0; n < kNt; ++n) {
                    float t[4];
                    mma16816_first<true>(t, a[0][0], a[1][0], a[0][1], a[1][1], q[n][2 * j][0], q[n][2 * j][1]);
                    mma16816<true>(t, a[0][2], a[1][2], a[0][3], a[1][3], q[n][2 * j + 1][0], q[n][2 * j + 1][1]);
                    const float2 w = make_float2(qs[n][j][0], qs[n][j][1]), base = make_float2(qa[n][j][0], qa[n][j][1]);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        sum[n][i] = j == 0 ? fmul2(mid[i], w) : ffma2(mid[i], w, sum[n][i]);
                        sum[n][i] = ffma2(scale[i], fadd2(make_float2(t[2 * i], t[2 * i + 1]), base), sum[n][i]);
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < kNt; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    s[n][2 * i] = sum[n][i].x;
                    s[n][2 * i + 1] = sum[n][i].y;
                }
        }
    }

    // Adds 16 keys' values with the weights s.
    __device__ __forceinline__ void values(const float (&s)[kNt][4], const uint8_t* sub, int g, int c) {
        KvRegs<HD, kBits> x;
        x.load_v(sub, g, c);
        if constexpr (kBits == 16) {
            uint32_t b[kNt][2], b2[kNt][2];
#pragma unroll
            for (int n = 0; n < kNt; ++n) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    // Toward 0, and what that leaves.  Neither part is 0, so that infinite values under any weight are
                    // infinities: f16 parts are 2^-24 at least, 2^-35 of the largest weight together, bf16 ones are not 0 where
                    // the fp32 weight is not (2^-126 of the largest).
                    if constexpr (kHalf) {
                        const float p0 = fmaxf(s[n][2 * i], 0x1p-24f), p1 = fmaxf(s[n][2 * i + 1], 0x1p-24f);
                        const uint32_t hi = pack_f16x2_rz(p0, p1);
                        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
                        b[n][i] = movmatrix_t(hi);
                        b2[n][i] = movmatrix_t(pack_f16x2(fmaxf(p0 - f.x, 0x1p-24f), fmaxf(p1 - f.y, 0x1p-24f)));
                    } else {
                        const float p0 = s[n][2 * i], p1 = s[n][2 * i + 1];
                        const uint32_t u = __float_as_uint(p0), w = __float_as_uint(p1);
                        b[n][i] = movmatrix_t(__byte_perm(u, w, 0x7632));
                        b2[n][i] = movmatrix_t(pack_bf16x2(fmaxf(p0 - __uint_as_float(u & 0xffff0000u), 1e-37f),
                                                           fmaxf(p1 - __uint_as_float(w & 0xffff0000u), 1e-37f)));
                    }
                }
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
                    for (int n = 0; n < kNt; ++n) {
                        mma16816<kHalf>(o[n][4 * j + t], a0, a1, a2, a3, b[n][0], b[n][1]);
                        mma16816<kHalf>(o[n][4 * j + t], a0, a1, a2, a3, b2[n][0], b2[n][1]);
                    }
                }
            }
        } else {
            uint32_t b[kNt][2], b2[kNt][2];
#pragma unroll
            for (int n = 0; n < kNt; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const __half2 hi = __floats2half2_rn(s[n][2 * i], s[n][2 * i + 1]);
                    b[n][i] = movmatrix_t(*reinterpret_cast<const uint32_t*>(&hi));
                    if constexpr (kSplitP) {
                        const float2 f = __half22float2(hi);
                        b2[n][i] = movmatrix_t(pack_f16x2(s[n][2 * i] - f.x, s[n][2 * i + 1] - f.y));
                    }
                }
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
                // [i]: keys 2c, 2c + 1, and 2c + 8, 2c + 9, beside each other
                __half2 v[2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t sp = __byte_perm(x.vp[2 * i][j], x.vp[2 * i + 1][j], 0x5410);
                    const uint32_t mp = __byte_perm(x.vp[2 * i][j], x.vp[2 * i + 1][j], 0x7632);
                    const __half2 scale = *reinterpret_cast<const __half2*>(&sp), mid = *reinterpret_cast<const __half2*>(&mp);
                    const uint32_t u = __byte_perm(x.v[2 * i][j / 2], x.v[2 * i + 1][j / 2], (j & 1) ? 0x7632 : 0x5410);
                    const uint32_t u8 = u >> 8;
                    v[i][0] = __hfma2(code_value<false>(u), scale, mid);
                    v[i][1] = __hfma2(code_value<true>(u), scale, mid);
                    v[i][2] = __hfma2(code_value<false>(u8), scale, mid);
                    v[i][3] = __hfma2(code_value<true>(u8), scale, mid);
                }
                const uint32_t(*a)[4] = reinterpret_cast<const uint32_t(*)[4]>(v);
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int n = 0; n < kNt; ++n) {
                        mma16816<true>(o[n][2 * j + t], a[0][2 * t], a[0][2 * t + 1], a[1][2 * t], a[1][2 * t + 1], b[n][0],
                                       b[n][1]);
                        if constexpr (kSplitP)
                            mma16816<true>(o[n][2 * j + t], a[0][2 * t], a[0][2 * t + 1], a[1][2 * t], a[1][2 * t + 1],
                                           b2[n][0], b2[n][1]);
                    }
            }
        }
    }

    // mid + scale (c - 8) may be past the largest fp16 though the group's values are not (up to 65568: both parameters and the
    // code are rounded).  Such keys have their V parameters halved in the stage and their weights doubled.
    // large_values: whether this lane's key of the stage may be one; what is left alone is under 49152 + 8 * 2048 in magnitude.
    // (One read, four comparisons and a share of the vote on the base: 76.3 -> 79.1 us at 4 sequences of up to 65536 tokens,
    // 14.1 -> 14.4 at 64 windows.  Clamping each value instead takes two instructions for every two of them.)
    static __device__ __forceinline__ uint8_t* v_params(uint8_t* stage, int lane) {
        using St = KvStage<HD, kBits>;
        return stage + (lane >> 4) * St::kSubBytes + St::kVp + (lane & 15) * St::kPar;
    }
    static __device__ __forceinline__ bool large_values(uint8_t* stage, int lane) {
        uint32_t w[kGroups];  // (scale, mid)
        load_words(w, v_params(stage, lane));
        const __half2* par = reinterpret_cast<const __half2*>(w);
        __half2 top = __hmax2(__habs2(par[0]), __habs2(par[1]));
        if constexpr (kGroups == 4) top = __hmax2(top, __hmax2(__habs2(par[2]), __habs2(par[3])));
        return !__hbltu2(top, __floats2half2_rn(2048.f, 49152.f));  // (a group that is NaN need not be one)
    }
    // (Halved, a subnormal parameter of another group of such a key is off by 2^-25.)
    static __device__ __forceinline__ void double_large(float (&s)[KvStage<HD, kBits>::kSub][kNt][4], uint8_t* stage,
                                                        int lane, uint32_t keys) {
        if ((keys >> lane) & 1) {
            __half2* par = reinterpret_cast<__half2*>(v_params(stage, lane));
#pragma unroll
            for (int j = 0; j < kGroups; ++j) par[j] = __hmul2(par[j], __float2half2_rn(0.5f));
        }
        __syncwarp();
        const int g = lane >> 2;
#pragma unroll
        for (int u = 0; u < KvStage<HD, kBits>::kSub; ++u)
#pragma unroll
            for (int n = 0; n < kNt; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if ((keys >> (16 * u + 8 * (i >> 1) + g)) & 1) s[u][n][i] *= 2.f;
    }

    // The A operands of value tile T (two dimensions of this lane): keys 2c, 2c + 1 beside each other, then 2c + 8, 2c + 9.
    static __device__ __forceinline__ void value_tile(const KvRegs<HD, kBits>& x, int T, uint32_t (&a)[4]) {
        if constexpr (kBits == 16) {
            const int j = T / 4, t = T % 4;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t v0 = (&x.v[2 * i][j].x)[t], v1 = (&x.v[2 * i + 1][j].x)[t];
                a[2 * i] = __byte_perm(v0, v1, 0x5410);
                a[2 * i + 1] = __byte_perm(v0, v1, 0x7632);
            }
        } else {
            const int j = T / 2;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t sp = __byte_perm(x.vp[2 * i][j], x.vp[2 * i + 1][j], 0x5410);
                const uint32_t mp = __byte_perm(x.vp[2 * i][j], x.vp[2 * i + 1][j], 0x7632);
                uint32_t u = __byte_perm(x.v[2 * i][j / 2], x.v[2 * i + 1][j / 2], (j & 1) ? 0x7632 : 0x5410);
                if (T & 1) u >>= 8;
                const __half2 scale = *reinterpret_cast<const __half2*>(&sp), mid = *reinterpret_cast<const __half2*>(&mp);
                const __half2 lo = __hfma2(code_value<false>(u), scale, mid), up = __hfma2(code_value<true>(u), scale, mid);
                a[2 * i] = *reinterpret_cast<const uint32_t*>(&lo);
                a[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&up);
            }
        }
    }

    // values() where not every row sees every key: weights of 0 are 0 in both parts, and where there are values that are no
    // numbers, the products are taken token by token.  key(i): code of key i of these 16 (KvTile::sees).
    template <typename Tile, typename Key>
    __device__ __forceinline__ void values_masked(const float (&s)[kNt][4], const uint8_t* sub, int g, int c,
                                                  const Tile& tile, Key key) {
        constexpr bool kF16 = kBits == 4 || kHalf, kTwo = kBits == 16 || kSplitP;
        KvRegs<HD, kBits> x;
        x.load_v(sub, g, c);
        uint32_t b[kNt][2], b2[kNt][2];
#pragma unroll
        for (int n = 0; n < kNt; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float p0 = s[n][2 * i], p1 = s[n][2 * i + 1];
                if constexpr (kHalf && kBits == 16) {
                    if (p0 != 0.f) p0 = fmaxf(p0, 0x1p-24f);
                    if (p1 != 0.f) p1 = fmaxf(p1, 0x1p-24f);
                }
                uint32_t hi;
                float2 f;
                if constexpr (kF16) {
                    hi = kTwo ? pack_f16x2_rz(p0, p1) : pack_f16x2(p0, p1);
                    f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
                } else {
                    hi = __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632);
                    f = make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u));
                }
                b[n][i] = movmatrix_t(hi);
                constexpr float kTiny = kF16 ? 0x1p-24f : 1e-37f;
                const float l0 = p0 == 0.f ? 0.f : fmaxf(p0 - f.x, kTiny), l1 = p1 == 0.f ? 0.f : fmaxf(p1 - f.y, kTiny);
                if constexpr (kTwo) b2[n][i] = movmatrix_t(kF16 ? pack_f16x2(l0, l1) : pack_bf16x2(l0, l1));
            }
        constexpr uint32_t kExp = kF16 ? 0x7c007c00u : 0x7f807f80u;
        bool odd = false;  // an exponent of all ones
#pragma unroll
        for (int T = 0; T < HD / 16; ++T) {
            uint32_t a[4];
            value_tile(x, T, a);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t e = ~a[i] & kExp;
                odd |= !(e & 0xffffu) || !(e >> 16);
            }
        }
        if (!__any_sync(~0u, odd)) {
#pragma unroll
            for (int T = 0; T < HD / 16; ++T) {
                uint32_t a[4];
                value_tile(x, T, a);
#pragma unroll
                for (int n = 0; n < kNt; ++n) {
                    mma16816<kF16>(o[n][T], a[0], a[1], a[2], a[3], b[n][0], b[n][1]);
                    if constexpr (kTwo) mma16816<kF16>(o[n][T], a[0], a[1], a[2], a[3], b2[n][0], b2[n][1]);
                }
            }
            return;
        }
        for (int t = 0; t < tile.rows; ++t) {  // token t's keys alone, into its own columns
            const int2 see = tile.row(t);
            uint32_t keep[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int k0 = key(2 * c + 8 * i), k1 = key(2 * c + 8 * i + 1);
                keep[i] = (Tile::sees(see, k0) ? 0xffffu : 0u) | (Tile::sees(see, k1) ? 0xffff0000u : 0u);
            }
#pragma unroll
            for (int T = 0; T < HD / 16; ++T) {
                uint32_t a[4];
                value_tile(x, T, a);
#pragma unroll
                for (int n = 0; n < kNt; ++n) {
                    float r[4];
                    mma16816_first<kF16>(r, a[0] & keep[0], a[1] & keep[0], a[2] & keep[1], a[3] & keep[1], b[n][0], b[n][1]);
                    if constexpr (kTwo)
                        mma16816<kF16>(r, a[0] & keep[0], a[1] & keep[0], a[2] & keep[1], a[3] & keep[1], b2[n][0], b2[n][1]);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if ((8 * n + 2 * c + (i & 1)) / tile.gs == t) o[n][T][i] += r[i];
                }
            }
        }
    }

    // One step over a stage; bit i of ok: there is a key i.  masked (kPack): not every row sees every key.
    template <typename Tile>
    __device__ __forceinline__ void step(uint8_t* stage, int g, int c, uint32_t ok, bool masked, int code,
                                         const Tile& tile) {
        constexpr int kSub = KvStage<HD, kBits>::kSub;
        constexpr uint32_t kAll = kSub == 2 ? ~0u : 0xffffu;
        float s[kSub][kNt][4];
        bool large = false;
        if constexpr (kBits == 4) large = large_values(stage, 4 * g + c);
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
            scores(s[u], stage + u * KvStage<HD, kBits>::kSubBytes, g, c);
#pragma unroll
            for (int n = 0; n < kNt; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[u][n][i] *= rs[n][i & 1];
        }
        if constexpr (kPack) {
            if (masked) {
                int k[kSub][2];
#pragma unroll
                for (int u = 0; u < kSub; ++u)
#pragma unroll
                    for (int i = 0; i < 2; ++i) k[u][i] = __shfl_sync(~0u, code, 16 * u + 8 * i + g);
#pragma unroll
                for (int n = 0; n < kNt; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int2 see = tile.row((8 * n + 2 * c + e) / tile.gs);
#pragma unroll
                        for (int u = 0; u < kSub; ++u)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                if (!Tile::sees(see, k[u][i])) s[u][n][2 * i + e] = -INFINITY;
                    }
            }
        } else if (ok != kAll) {
#pragma unroll
            for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (!((ok >> (16 * u + 8 * i + g)) & 1))
#pragma unroll
                        for (int n = 0; n < kNt; ++n) s[u][n][2 * i] = s[u][n][2 * i + 1] = -INFINITY;
        }
        // The exponent base moves only when a score exceeds it by more than
        // kRoom (or there is none yet).
        float top[kNt][2];
        bool move = large;
        uint32_t keys = 0;  // 4 bits: those of large values
#pragma unroll
        for (int n = 0; n < kNt; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                top[n][e] = fmaxf(s[0][n][e], s[0][n][2 + e]);
                if constexpr (kSub == 2) top[n][e] = fmaxf(top[n][e], fmaxf(s[kSub - 1][n][e], s[kSub - 1][n][2 + e]));
                move |= top[n][e] > m[n][e] + kRoom;
            }
        if (__any_sync(~0u, move)) {
            if constexpr (kBits == 4) keys = __ballot_sync(~0u, large);
#pragma unroll
            for (int n = 0; n < kNt; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float t = fmaxf(m[n][e], top[n][e]);
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
                }
        }
#pragma unroll
        for (int n = 0; n < kNt; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float base = m[n][e] == -INFINITY ? 0.f : m[n][e] - kLift;  // no score but -inf yet: weights of 0
#pragma unroll
                for (int u = 0; u < kSub; ++u)
#pragma unroll
                    for (int i = e; i < 4; i += 2) {
                        s[u][n][i] = ex2_approx(s[u][n][i] - base);
                        l[n][e] += s[u][n][i];
                    }
            }
        if constexpr (kBits == 4)
            if (keys) double_large(s, stage, 4 * g + c, keys);
        if constexpr (kPack)
            if (masked) {
#pragma unroll
                for (int u = 0; u < kSub; ++u)
                    values_masked(s[u], stage + u * KvStage<HD, kBits>::kSubBytes, g, c, tile,
                                  [&](int i) { return __shfl_sync(~0u, code, 16 * u + i); });
                return;
            }
#pragma unroll
        for (int u = 0; u < kSub; ++u) values(s[u], stage + u * KvStage<HD, kBits>::kSubBytes, g, c);
    }
};

// The rows of a unit's tile and what they see.  A key's code: its position j for
// one of the window's block, ~j for an entry of the global list, kNoKey for none.
constexpr int kNoKey = 0x7fffffff;
struct KvTile {
    int pos, r, rows, globals, gs;
    // Row t's window, first and last key; (0, -1) of a row that is none.
    __device__ __forceinline__ int2 row(int t) const {
        return t < rows ? make_int2((globals >> t) & 1 ? 0 : max(0, pos + t - r), pos + t) : make_int2(0, -1);
    }
    // Window keys of the row's own window, list entries below it.
    static __device__ __forceinline__ bool sees(int2 row, int code) {
        return code >= 0 ? code >= row.x && code <= row.y : ~code < row.x;
    }
};

// Where a CTA is in its range of the work sequence; all warps walk alike.
template <int block, bool kPack>
struct KvWalk {
    int row, unit, seq, pos, ng, lo, tile, head;
    int b, b1, nb;   // the next block of the unit, and where the CTA's piece of it ends
    int64_t left;    // of the range from block b on
    KvKeys u;

    __device__ __forceinline__ void enter(const KvAttnParams& p) {
        head = unit / p.nsub;
        u = kPack ? KvKeys(lo, pos + (tile & 255) - 1, ng) : KvKeys(pos, ng, p.r, p.dil[head]);
        nb = u.blocks(block);
        b1 = static_cast<int>(min(int64_t(nb), b + left));
    }
    __device__ __forceinline__ KvWalk(const KvAttnParams& p, const KvStart& s)
        : row(s.row), unit(s.unit), seq(s.seq), pos(s.pos), ng(s.ng), lo(s.lo), tile(s.tile), b(s.blk), left(s.n),
          u(0, 0, 0) {
        enter(p);
    }
    __device__ __forceinline__ void next_unit(const KvAttnParams& p) {
        b = 0;
        if (++unit == p.kv_heads * p.nsub) {
            unit = 0;
            do ++row;
            while (row < p.N && p.plan.row_tile[row] == 0);  // rows that begin no tile
            if (row >= p.N) {
                left = 0;
                return;
            }
            seq = p.plan.row_seq[row];
            pos = p.plan.row_pos[row];
            ng = p.plan.row_ng[row];
            if constexpr (kPack) {
                lo = p.plan.row_lo[row];
                tile = p.plan.row_tile[row];
            }
        }
        left -= kUnitKeys / block;
        enter(p);
    }

    // Whether some row does not see some of the warp's keys of block b (kPack).
    __device__ __forceinline__ bool masked(const KvAttnParams& p, int warp) const {
        const int n0 = b * block + block / kKvWarps * warp, n1 = n0 + block / kKvWarps, last = pos + (tile & 255) - 1;
        return n1 > u.n_win || u.first + n1 - 1 > pos || u.first + n0 < max(0, last - p.r);
    }

    // The row of the cache that key i = lane % (keys of a warp) of the warp's part of block b is in, -1: no such key;
    // and its code (KvTile).
    __device__ __forceinline__ int key_row(const KvAttnParams& p, int warp, int lane, int& code) const {
        constexpr int kKeys = block / kKvWarps;
        const int n = b * block + kKeys * warp + (lane & (kKeys - 1));
        code = kNoKey;
        if (n >= u.n) return -1;
        int at;
        if (n < u.n_win) {
            at = u.first + n * u.step;
        } else {
            at = p.plan.g_list[int64_t(seq) * p.n_global + (n - u.n_win)];
            if constexpr (!kPack) {
                const int back = pos - at;  // > 0
                if (back % u.step == 0 && back / u.step < u.n_win) return -1;  // in the window
            }
        }
        const int page = p.table[int64_t(seq) * p.max_pages + (at >> p.log_page)];
        if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.n_pages)) {
            atomicOr(p.status, kStatusBadCache);
            return -1;
        }
        code = n < u.n_win ? at : ~at;
        return ((page * p.kv_heads + head) << p.log_page) + (at & ((1 << p.log_page) - 1));
    }
};

template <bool kHalf>
__device__ __forceinline__ void store16(void* at, int64_t i, float x) {
    if constexpr (kHalf) static_cast<__half*>(at)[i] = __float2half_rn(x);
    else static_cast<__nv_bfloat16*>(at)[i] = __float2bfloat16_rn(x);
}

// Floats of a partial state: O, m and l of each query row of a unit, in whole 16 bytes.
__host__ __device__ constexpr int kv_piece_row(int d) { return d + 4; }

// The warps' rings, and room to join 8 query rows' 64 dimensions of the four warps at a time: a row of 68 floats, so
// that the 16-byte stores of eight lanes (four rows, two places) meet all banks.
constexpr int kJoinRow = 68;
template <int HD, int kBits>
constexpr int kv_attn_smem(int unit_rows) {
    return kKvWarps * (kStages * KvStage<HD, kBits>::kBytes + (unit_rows < 8 ? unit_rows : 8) * kJoinRow * 4);
}

template <int HD, int kBits, bool kHalf, int kNt, bool kPack>
__global__ void __launch_bounds__(kKvThreads, kv_ctas_per_sm(HD, kBits, kNt == 2, kPack))
    kv_attn_kernel(const __grid_constant__ KvAttnParams p) {
    constexpr int kRows = 8 * kNt;
    constexpr int kStage = KvStage<HD, kBits>::kBytes;
    constexpr int kBlock = kv_block(kBits);
    constexpr int kUnits = 8;  // descriptors in flight: at most kStages + 2 units are between the walk and the end
    using State = KvState<HD, kBits, kHalf, kNt, kPack>;
    extern __shared__ __align__(128) uint8_t s_ring[];
    float* s_o = reinterpret_cast<float*>(s_ring + kKvWarps * kStages * kStage);
    __shared__ float s_m[kKvWarps][kRows], s_l[kKvWarps][kRows];
    __shared__ int4 s_unit[kKvWarps][kUnits];  // row, unit, tile, slot of its partial state (-1: whole)
    __shared__ int s_pos[kKvWarps][kUnits];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int s = blockIdx.x;
    grid_dep_launch();
    const KvStart start = p.plan.start[s];  // (at a fixed place of any plan)
    if (p.plan.sig[1] != p.sig) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusBadPlan);
        return;
    }
    if (start.n <= 0) return;
    uint8_t* ring = s_ring + warp * (kStages * kStage);
    const uint32_t ring_at = smem_u32(ring);

    // The walk runs ahead of the blocks that are computed.  Of each block in
    // flight: which of the warp's keys there are (kPack: their codes), and a
    // note: bit 0 first and bit 1 last of its piece, bit 2 masked, bits 3 to 5
    // the unit's descriptor, bit 6 that there is a block.
    KvWalk<kBlock, kPack> w(p, start);
    int entered = 0;
    auto describe = [&](bool first_piece) {
        const bool whole = w.b == 0 && w.b1 == w.nb;
        // slot 2s: the piece a CTA begins with, of a unit that an earlier one began; 2s + 1: one that a later CTA ends
        if (lane == 0) {
            s_unit[warp][entered % kUnits] =
                make_int4(w.row, w.unit, w.tile, whole ? -1 : 2 * s + (first_piece && w.b > 0 ? 0 : 1));
            if constexpr (kPack) s_pos[warp][entered % kUnits] = w.pos;
        }
    };
    int row_next = -1, code_next = kNoKey;
    uint32_t note_next = 0;
    bool fresh = true;
    describe(true);
    auto fetch = [&] {
        row_next = -1;
        note_next = 0;
        if (w.left <= 0) return;
        row_next = w.key_row(p, warp, lane, code_next);
        note_next = (fresh ? 1u : 0u) | (w.b + 1 == w.b1 ? 2u : 0u) | uint32_t(entered % kUnits) << 3 | 64u;
        if constexpr (kPack) note_next |= w.masked(p, warp) ? 4u : 0u;
        fresh = false;
        --w.left;
        if (++w.b == w.b1 && w.left > 0) {
            w.next_unit(p);
            ++entered;
            fresh = true;
            describe(false);
        }
    };
    uint32_t ok[kStages], note[kStages];
    int code[kStages];
    auto issue = [&](int stage, int i) {
        kv_issue<HD, kBits>(p, ring_at + stage * kStage, row_next, lane);
        cp_async_commit();
        ok[i] = __ballot_sync(~0u, row_next >= 0) & (kBlock == 64 ? 0xffffu : ~0u);
        note[i] = note_next;
        code[i] = code_next;
        if (kPack && ok[i] != (kBlock == 64 ? 0xffffu : ~0u)) note[i] |= 4u;
    };
    fetch();
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
        issue(i, i);
        fetch();
    }
    auto query = [&](uint4 (&x)[kNt][HD / 32], uint32_t m) {
        const int4 d = s_unit[warp][(m >> 3) & 7];
        const int head = d.y / p.nsub, sub = d.y - head * p.nsub;
        State::load_q(x, p, static_cast<const uint8_t*>(p.q) + 2 * (d.x * p.q_row + (head * p.group + sub * p.gs) * p.q_head),
                      kPack ? (d.z & 255) * p.gs : min(p.gs, p.group - sub * p.gs), lane);
    };
    State st;
    uint4 qn[kNt][HD / 32];
    __syncwarp();
    query(qn, note[0]);
    int stage = 0;
    while (note[0] & 64u) {
        __syncwarp();  // every lane has read the stage that is filled next
        issue(stage == 0 ? kStages - 1 : stage - 1, kStages - 1);
        fetch();
        const uint32_t now = note[0];
        if (now & 1u) st.begin(qn, lane, p.sl2);
        __syncwarp();
        if (note[1] & 1u) query(qn, note[1]);
        cp_async_wait<kStages - 1>();
        __syncwarp();
        if constexpr (kPack) {
            const int z = s_unit[warp][(now >> 3) & 7].z;
            const KvTile tile{s_pos[warp][(now >> 3) & 7], p.r, z & 255, z >> 8, p.gs};
            if (ok[0]) st.step(ring + stage * kStage, g, c, ok[0], now & 4u, code[0], tile);
        } else {
            if (ok[0]) st.step(ring + stage * kStage, g, c, ok[0], false, 0, 0);
        }
        if (now & 2u) {  // join the lanes' and the warps' states
            const int4 d = s_unit[warp][(now >> 3) & 7];
            const int head = d.y / p.nsub, sub = d.y - head * p.nsub;
            const int rows = kPack ? (d.z & 255) * p.gs : min(p.gs, p.group - sub * p.gs), qh = head * p.group + sub * p.gs;
            const int join = min(p.unit_rows, 8) * kJoinRow;  // floats of a warp
            float* part = p.part + int64_t(d.w) * p.unit_rows * kv_piece_row(HD);
#pragma unroll
            for (int n = 0; n < kNt; ++n) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float l = st.l[n][e];
                    l += __shfl_xor_sync(~0u, l, 4);
                    l += __shfl_xor_sync(~0u, l, 8);
                    l += __shfl_xor_sync(~0u, l, 16);
                    if (g == 0) {
                        s_m[warp][8 * n + 2 * c + e] = st.m[n][e];
                        s_l[warp][8 * n + 2 * c + e] = l;
                    }
                }
#pragma unroll
                for (int half = 0; half < HD / 64; ++half) {
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (8 * n + 2 * c + e < rows) {
                            float* at = s_o + warp * join + (2 * c + e) * kJoinRow;
                            float4 x[2];
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                x[k] = make_float4(st.o[n][4 * half + 2 * k][e], st.o[n][4 * half + 2 * k][2 + e],
                                                   st.o[n][4 * half + 2 * k + 1][e], st.o[n][4 * half + 2 * k + 1][2 + e]);
                            if constexpr (kBits == 16) {  // odd g in the other order: eight lanes meet all banks
                                const bool odd = g & 1;
                                *reinterpret_cast<float4*>(at + 8 * g + (odd ? 4 : 0)) = odd ? x[1] : x[0];
                                *reinterpret_cast<float4*>(at + 8 * g + (odd ? 0 : 4)) = odd ? x[0] : x[1];
                            } else {
                                *reinterpret_cast<float4*>(at + 4 * g) = x[0];
                                *reinterpret_cast<float4*>(at + 32 + 4 * g) = x[1];
                            }
                        }
                    __syncthreads();
                    // a thread takes four dimensions of a row (once; as a loop the blocks' code comes out 3 % faster)
                    for (int i = threadIdx.x; i < 16 * min(8, rows - 8 * n); i += kKvThreads) {
                        const int r = i / 16, h = 8 * n + r, e = 4 * (i % 16);
                        float m = s_m[0][h];
#pragma unroll
                        for (int a = 1; a < kKvWarps; ++a) m = fmaxf(m, s_m[a][h]);
                        float l = 0.f;
                        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int a = 0; a < kKvWarps; ++a) {
                            // a warp without keys has m = -inf and zeros
                            const float f = s_m[a][h] == m ? 1.f : ex2_approx(s_m[a][h] - m);
                            const float4 y = *reinterpret_cast<const float4*>(s_o + a * join + r * kJoinRow + e);
                            l += s_l[a][h] * f;
                            o.x += y.x * f;
                            o.y += y.y * f;
                            o.z += y.z * f;
                            o.w += y.w * f;
                        }
                        if (d.w < 0) {
                            const int64_t at = d.x * p.o_row + qh * p.o_head + State::row_at(h, p.gs, p.o_row, p.o_head) +
                                               64 * half + e;
                            const float inv = l == 0.f ? 0.f : 1.f / l;
                            o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
                            if (p.o_wide) {
                                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) =
                                    kHalf ? make_uint2(pack_f16x2(o.x, o.y), pack_f16x2(o.z, o.w))
                                          : make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
                            } else {
                                store16<kHalf>(p.out, at, o.x);
                                store16<kHalf>(p.out, at + 1, o.y);
                                store16<kHalf>(p.out, at + 2, o.z);
                                store16<kHalf>(p.out, at + 3, o.w);
                            }
                        } else {
                            float* at = part + h * kv_piece_row(HD);
                            *reinterpret_cast<float4*>(at + 64 * half + e) = o;
                            if (half == 0 && e == 0) {
                                at[HD] = m;
                                at[HD + 1] = l;
                            }
                        }
                    }
                    __syncthreads();
                }
            }
        }
#pragma unroll
        for (int i = 0; i + 1 < kStages; ++i) {
            ok[i] = ok[i + 1];
            note[i] = note[i + 1];
            code[i] = code[i + 1];
        }
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    cp_async_wait<0>();
}

// Joins the pieces of the unit that CTA s of the attention began and CTA
// cut.last ended: y = sum of 2^(m_k - M) O_k over sum of 2^(m_k - M) l_k, M =
// max m_k, in CTA order.  grid: (G, query rows of a unit), HD threads, one
// per dimension; the attention's programmatic dependent.  Bound: latency (all
// pieces' m and l at once, then their O eight at a time: 6 us with its launch;
// one piece after the other took 49 us at 12 pieces of 8 heads).  A grid of
// cut units alone, listed by the plan, measured 0.9 us slower.
template <int HD, bool kHalf>
__global__ void __launch_bounds__(HD) kv_merge_kernel(const __grid_constant__ KvAttnParams p) {
    __shared__ float s_w[HD], s_red[2];
    const int s = blockIdx.x, h = blockIdx.y, e = threadIdx.x;
    const KvCut cut = p.plan.cut[s];
    const bool mine = cut.last >= 0 && p.plan.sig[1] == p.sig;
    grid_dep_wait();
    if (!mine) return;
    const int head = cut.unit / p.nsub, sub = cut.unit - head * p.nsub;
    const bool pack = p.unit_rows > p.gs;
    const int rows = pack ? (cut.tile & 255) * p.gs : min(p.gs, p.group - sub * p.gs), qh = head * p.group + sub * p.gs;
    if (h >= rows) return;
    const int64_t at = cut.row * p.o_row + qh * p.o_head + (pack ? h / p.gs * p.o_row + h % p.gs * p.o_head : h * p.o_head);
    // piece 0 is in slot 2s + 1, piece k > 0 in slot 2 (s + k)
    const int64_t row = kv_piece_row(HD), piece = p.unit_rows * row;
    const float* base = p.part + 2 * int64_t(s) * piece + h * row;
    const int n = cut.last - s + 1;
    float M = -INFINITY, L = 0.f, O = 0.f;
    for (int k0 = 0; k0 < n; k0 += HD) {  // HD pieces at a time
        const int k = k0 + e;
        const float* a = base + (k == 0 ? piece : 2 * k * piece);
        const float m = k < n ? __ldcg(a + HD) : -INFINITY, l = k < n ? __ldcg(a + HD + 1) : 0.f;
        float t = m;
#pragma unroll
        for (int o = 16; o; o >>= 1) t = fmaxf(t, __shfl_xor_sync(~0u, t, o));
        if (e == 0) s_red[0] = M;
        __syncthreads();
        s_w[e] = t;  // each warp's maximum, in all its lanes' places
        __syncthreads();
        float top = s_red[0];
#pragma unroll
        for (int a = 0; a < HD / 32; ++a) top = fmaxf(top, s_w[32 * a]);
        __syncthreads();
        const float f = m == top ? 1.f : ex2_approx(m - top);
        s_w[e] = k < n ? f : 0.f;
        float ls = k < n ? l * f : 0.f;
        const float old = M == top ? 1.f : ex2_approx(M - top);
        O *= old;
        L *= old;
        M = top;
        __syncthreads();
        const int cnt = min(HD, n - k0);
#pragma unroll 8
        for (int i = 0; i < cnt; ++i) {
            const int kk = k0 + i;
            O += s_w[i] * __ldcg(base + (kk == 0 ? piece : 2 * kk * piece) + e);
        }
        // the sum, over the threads in a fixed order
        __syncthreads();
        s_w[e] = ls;
        __syncthreads();
        for (int i = 0; i < cnt; ++i) L += s_w[i];
        __syncthreads();
    }
    store16<kHalf>(p.out, at + e, L == 0.f ? 0.f : O / L);
}

}  // namespace lf
