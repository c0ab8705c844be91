// kv_append.cuh -- a step's new tokens into the paged cache: the keys turned
// by their positions (rotary.cuh), the values as they are, both in 16 bits or
// quantised to 4; the queries turned beside them into dense rows, and, where
// the caller asks for them, the values that the cache now holds.
//
// 4 bits (groups of 32 values x of the row, in the 16-bit type):
//   scale = fp16((max - min) / 15), mid = fp16(min + 8 scale),
//   c = clamp(round((x - mid) / scale) + 8, 0, 15)   (ties to even; 8 if scale is 0)
// and the group stands for mid + scale (c - 8).  A group with a value past
// fp16's range, an infinity or a NaN is held as NaN (mid).
// Near a border between codes the subtraction and the division are IEEE ones,
// so that the codes are the formula's.
//
// Bound: bytes, as rotary.cuh.  For 4 bits a CTA's turned rows pass through
// shared memory (16-bit), where four neighbouring lanes take the 32 values
// of a group: its minimum and maximum are two shuffles, and each lane's codes
// make one 32-bit word of a K row and one unit of a V row for each of two
// lanes, exchanged so that both store whole words.  (Prompts of 4099 tokens,
// 36 rows of 64, 16 bits: 9.6 us, 3.9 TB/s, and 11.1 where nothing is in L2;
// 16384 tokens of 32 rows, 4 bits and what they hold: 42 us, 3.4 TB/s, 20 of
// them for the codes, which instructions bound.)
#pragma once
#include <type_traits>

#include "kv_plan.cuh"
#include "rotary.cuh"

namespace lf {

struct KvAppendParams {
    const void* x[3];  // k, v, q rows [N][heads][d]; q may be absent
    void* y[3];        // dense copies: held k, held v (may be absent), turned q
    int xt[3], xh[3];  // token and head strides, elements
    int yt[3], yh[3];
    int heads[3];
    uint8_t* cache[2];  // k, v
    uint8_t* par[2];    // 4 bits
    const int32_t* table;
    KvPlan plan;
    uint32_t* status;
    const double* freqs;  // null: no turn (rot == 0)
    int N, d, rot, n_pages, log_page, max_pages, inter;
    int log_tile, per;
    int wide;          // rows of x and y begin at 16-byte boundaries
    float amp;
    uint64_t sig;
};

// A tile's tokens: whether they are one, and the row of the cache of their kv
// head 0 (head h's is h pages' rows further), -1: none.
struct KvSlots {
    int live[kRotMaxTile], row[kRotMaxTile];
};

// Minimum and maximum of 8 values of a 16-bit type, pairwise; NaN if there is one.
template <typename T>
__device__ __forceinline__ void range8(uint4 x, float& lo, float& hi) {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    const T2* v = reinterpret_cast<const T2*>(&x);
    T2 a = __hmin2_nan(__hmin2_nan(v[0], v[1]), __hmin2_nan(v[2], v[3]));
    T2 b = __hmax2_nan(__hmax2_nan(v[0], v[1]), __hmax2_nan(v[2], v[3]));
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
        a = __hmin2_nan(a, __shfl_xor_sync(~0u, a, o));
        b = __hmax2_nan(b, __shfl_xor_sync(~0u, b, o));
    }
    a = __hmin2_nan(a, __lowhigh2highlow(a));
    b = __hmax2_nan(b, __lowhigh2highlow(b));
    lo = float(a.x);
    hi = float(b.x);
}

// Four lanes (lane & 3 = cc) hold the 32 values of group gr of a row, eight
// each (raw); all lanes of the warp take part, `on` ones have somewhere to
// put codes and parameters.  Gives the eight codes - 8, scale and mid.
// (x - mid) / scale clamped to a code and rounded: u = (x - mid) / (15 scale) +
// 8 / 15 saturates to 0..1 and 15 u is rounded by adding 1.5 * 2^23.  15 u is
// off by under 2^-18 (the reciprocal, its fifteenth, the sum, its constant),
// and only where it is that close to a border the group divides.
template <typename T>
__device__ __forceinline__ void quantise8(uint4 raw, bool is_k, bool on, int cc, int gr, int groups, uint8_t* codes,
                                          uint8_t* par, float& scale, float& mid, float (&c8)[8]) {
    float lo, hi, x[8];
    range8<T>(raw, lo, hi);
    RowIo<T>::widen(&raw, x);
    const __half hs = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f));
    scale = __half2float(hs);
    __half hm = __float2half_rn(__fadd_rn(lo, __fmul_rn(8.f, scale)));
    if (!(lo >= -65504.f && hi <= 65504.f)) hm = __float2half_rn(NAN);
    mid = __half2float(hm);
    const float inv = scale > 0.f ? __fdividef(1.f, 15.f * scale) : 0.f;  // scale 0: all codes 8
    constexpr float kRound = 12582912.f;
    uint32_t w = 0;
    float off = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float u = __saturatef(fmaf(__fsub_rn(x[i], mid), inv, 8.f / 15.f));
        const float r = fmaf(u, 15.f, kRound);
        const float whole = r - kRound;
        off = fmaxf(off, fabsf(fmaf(u, 15.f, -whole)));
        c8[i] = whole - 8.f;
        w += (__float_as_uint(r) - __float_as_uint(kRound)) << (4 * i);
    }
    if (off > 0.5f - 1.f / 131072.f && scale > 0.f) {
        w = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = rintf(__fdiv_rn(__fsub_rn(x[i], mid), scale)) + 8.f;
            const float c = fminf(fmaxf(q, 0.f), 15.f);
            c8[i] = c - 8.f;
            w |= static_cast<uint32_t>(c) << (4 * i);
        }
    }
    // V: units [r][g], r = 2 cc (low half of w) and 2 cc + 1; the lane of the neighbouring
    // group (lane ^ 4) has theirs: the even group stores unit r = 2 cc of both, the odd one 2 cc + 1
    const uint32_t other = __shfl_xor_sync(~0u, w, 4);
    if (!on) return;
    if (is_k) {
        reinterpret_cast<uint32_t*>(codes)[cc * groups + gr] = w;
    } else {
        const uint32_t pair = (gr & 1) ? __byte_perm(other, w, 0x7632) : __byte_perm(w, other, 0x5410);
        reinterpret_cast<uint32_t*>(codes)[((2 * cc + (gr & 1)) * groups + (gr & ~1)) / 2] = pair;
    }
    if (cc == 0)
        reinterpret_cast<uint32_t*>(par)[gr] =
            uint32_t(__half_as_ushort(hs)) | uint32_t(__half_as_ushort(hm)) << 16;
}

// Eight values that the cache now holds to a dense row.  f16: those past its range (up to 65568, where the group's ends
// are +-65504) as the nearest finite one; NaN stays NaN.
template <typename T>
__device__ __forceinline__ void store_held(T* y, const float (&x)[8], bool wide) {
    if constexpr (std::is_same<T, __half>::value) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("cvt.rn.satfinite.f16x2.f32 %0, %2, %1;" : "=r"(w[i]) : "f"(x[2 * i]), "f"(x[2 * i + 1]));
        if (wide) *reinterpret_cast<uint4*>(y) = make_uint4(w[0], w[1], w[2], w[3]);
        else
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = __ushort_as_half(static_cast<unsigned short>(w[i / 2] >> (16 * (i & 1))));
    } else {
        if (wide) RowIo<T>::store8(y, x);
        else
#pragma unroll
            for (int i = 0; i < 8; ++i) RowIo<T>::store(y + i, x[i]);
    }
}

// kW as in rotary_kernel.  grid: (tiles of tokens, 1 or 3): with 3 a CTA takes k, v or q only, where
// tiles alone are too few to fill the GPU.  smem: (cos, sin) [tile][cs_stride]; 4 bits: the
// turned k and v rows [k heads + v heads][tile][d] in 16 bits.
template <typename T, int kBits, int kW>
__global__ void __launch_bounds__(kRotThreads, kRotCtas) kv_append_kernel(const __grid_constant__ KvAppendParams p) {
    extern __shared__ __align__(16) uint8_t s_raw[];
    __shared__ KvSlots sl;
    if (p.plan.sig[0] != p.sig) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusBadPlan);
        return;
    }
    const int tile = 1 << p.log_tile, n0 = blockIdx.x * tile;
    const int nt = min(tile, p.N - n0), half = p.rot / 2, stride = cs_stride(half), kv = p.heads[0];
    float2* s_cs = reinterpret_cast<float2*>(s_raw);
    T* s_row = reinterpret_cast<T*>(s_raw + size_t(tile) * stride * 8);
    const int w0 = gridDim.y == 1 ? 0 : blockIdx.y, w1 = gridDim.y == 1 ? 3 : w0 + 1;
    auto ready = [&] {
        if (threadIdx.x < nt) {
            const int t = threadIdx.x, seq = p.plan.row_seq[n0 + t], pos = p.plan.row_pos[n0 + t];
            int row = -1;
            if (seq >= 0) {
                const int page = p.table[int64_t(seq) * p.max_pages + (pos >> p.log_page)];
                if (static_cast<unsigned>(page) < static_cast<unsigned>(p.n_pages))
                    row = ((page * kv) << p.log_page) + (pos & ((1 << p.log_page) - 1));
                else
                    atomicOr(p.status, kStatusBadCache);
            }
            sl.live[t] = seq >= 0;
            sl.row[t] = row;
        }
        for (int i = threadIdx.x; w0 != 1 && i < nt * half; i += kRotThreads) {
            const int t = i / half, f = i - t * half;
            s_cs[t * stride + cs_at(f, half)] = turn_of(p.plan.row_pos[n0 + t], p.freqs[f], p.amp, false);
        }
        __syncthreads();
    };
    // thread i has item i % per of token i / per % tile, and every step-th head
    const int rest = threadIdx.x / p.per, t = rest & (tile - 1), group = rest >> p.log_tile, it = threadIdx.x - rest * p.per;
    const int step = (kRotThreads / p.per) >> p.log_tile;
    int e0, e1;
    bool live = false;  // a row behind the last sequence stays as it was
    int row = -1;
    // Where head h of w (k, v, q) goes: q to its dense row, k and v to the cache (or to shared memory,
    // to be quantised) and, if asked for, to a dense row too.
    auto to = [&](int w, int h, T*(&dst)[2]) {
        dst[0] = dst[1] = nullptr;
        if ((w == 2 || kBits == 16) && p.y[w])
            dst[1] = static_cast<T*>(p.y[w]) + int64_t(n0 + t) * p.yt[w] + int64_t(h) * p.yh[w];
        if (w < 2) {
            if (kBits == 4) dst[0] = s_row + (((w * kv + h) << p.log_tile) + t) * p.d;
            else if (row >= 0) dst[0] = reinterpret_cast<T*>(p.cache[w]) + int64_t(row + (h << p.log_page)) * p.d;
        }
    };
    if constexpr (kW == 0) {
        item_at(it, p.rot, p.inter, e0, e1);
        float2 cs[8];
#pragma unroll 1
        for (int w = w0; w < w1; ++w) {
            if (p.heads[w] == 0) continue;
            move_rows<T>(
                static_cast<const T*>(p.x[w]) + int64_t(n0 + t) * p.xt[w], p.xh[w],
                group < step && t < nt ? group : p.heads[w], step, p.heads[w], e0, e1,
                [&] {
                    if (w > w0) return;  // there are always keys
                    ready();
                    if (t < nt) {
                        live = sl.live[t];
                        row = sl.row[t];
                        if (16 * it < p.rot) load_cs(cs, s_cs + t * stride, it, half);
                    }
                },
                [&](int h, float(&u)[8], float(&v)[8]) {
                    if (!live) return;
                    if (w != 1) turn_item(u, v, it, p.rot, p.inter, cs);
                    T* dst[2];
                    to(w, h, dst);
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (dst[k]) {
                            RowIo<T>::store8(dst[k] + e0, u);
                            RowIo<T>::store8(dst[k] + e1, v);
                        }
                });
        }
    } else {
        pair_at<kW>(it, p.d, p.rot, p.inter, e0, e1);  // (d is a multiple of 4: e1 is there)
        const bool turned = kW * it < half;
        float2 cs[kW];
#pragma unroll 1
        for (int w = w0; w < w1; ++w) {
            if (p.heads[w] == 0) continue;
            move_pairs<T, kW>(
                static_cast<const T*>(p.x[w]) + int64_t(n0 + t) * p.xt[w], p.xh[w],
                group < step && t < nt ? group : p.heads[w], step, p.heads[w], e0, e1,
                [&] {
                    if (w > w0) return;  // there are always keys
                    ready();
                    if (t < nt) {
                        live = sl.live[t];
                        row = sl.row[t];
                        if (turned)
#pragma unroll
                            for (int i = 0; i < kW; ++i) cs[i] = s_cs[t * stride + cs_at(kW * it + i, half)];
                    }
                },
                [&](int h, float(&u)[kW], float(&v)[kW]) {
                    if (!live) return;
                    if (w != 1 && turned)
#pragma unroll
                        for (int i = 0; i < kW; ++i) turn_pair(u[i], v[i], cs[i]);
                    T* dst[2];
                    to(w, h, dst);
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (dst[k]) {
                            store_few<T, kW>(dst[k] + e0, u);
                            store_few<T, kW>(dst[k] + e1, v);
                        }
                });
        }
    }
    if constexpr (kBits == 4) {
        __syncthreads();
        const int groups = p.d / 32, log_chunks = p.d == 64 ? 3 : 4, ch = threadIdx.x & ((1 << log_chunks) - 1);
#pragma unroll 1
        for (int w = w0; w < min(w1, 2); ++w) {
            const int rows = kv << p.log_tile;  // a warp has whole rows: 8 or 16 lanes each
            for (int i0 = 0; i0 < rows; i0 += kRotThreads >> log_chunks) {
                const int i = i0 + (threadIdx.x >> log_chunks), a = i & (tile - 1), h = i >> p.log_tile;
                const bool mine = i < rows && a < nt && sl.live[a];
                const uint4 raw = mine ? *reinterpret_cast<const uint4*>(s_row + (w * rows + i) * p.d + 8 * ch)
                                       : make_uint4(0, 0, 0, 0);
                const int r = mine ? sl.row[a] : -1;
                const int64_t at = r < 0 ? 0 : r + (h << p.log_page);
                float scale, mid, c8[8];
                quantise8<T>(raw, w == 0, r >= 0, ch & 3, ch >> 2, groups, p.cache[w] + at * (p.d / 2),
                             p.par[w] + at * (4 * groups), scale, mid, c8);
                if (mine && p.y[w]) {
                    T* y = static_cast<T*>(p.y[w]) + int64_t(n0 + a) * p.yt[w] + int64_t(h) * p.yh[w] + 8 * ch;
#pragma unroll
                    for (int k = 0; k < 8; ++k) c8[k] = fmaf(scale, c8[k], mid);
                    store_held<T>(y, c8, p.wide);
                }
            }
        }
    }
}

}  // namespace lf
