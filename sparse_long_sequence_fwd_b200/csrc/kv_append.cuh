// kv_append.cuh -- a step's new tokens into the paged cache: the keys turned
// by their positions (rotary.cuh), the values as they are, both in 16 bits or
// quantised to 4; the queries turned beside them into dense rows, and, where
// the caller asks for them, the values that the cache now holds.
//
// 4 bits (groups of 32 values x of the row, in the 16-bit type):
//   scale = fp16((max - min) / 15), mid = fp16(min + 8 scale),
//   c = clamp(round((x - mid) / scale) + 8, 0, 15)   (ties to even; 8 if scale is 0)
// and the group stands for mid + scale (c - 8).  A group with an infinity or
// a NaN is held as NaN (mid).  Near a border between codes the subtraction
// and the division are IEEE ones, so that the codes are the formula's.
//
// Bound: bytes, as rotary.cuh.  For 4 bits a CTA's turned rows pass through
// shared memory (16-bit), where four neighbouring lanes take the 32 values
// of a group: its minimum and maximum are two shuffles, and each lane's codes
// make one 32-bit word of a K row and one unit of a V row for each of two
// lanes, exchanged so that both store whole words.
#pragma once
#include <type_traits>

#include "kv_plan.cuh"
#include "rotary.cuh"

namespace lf {

struct KvAppendParams {
    const void* x[3];  // k, v, q rows [N][heads][d]; q may be absent
    int64_t xs[3][2];  // (token, head), elements
    void* y[3];        // dense copies: held k, held v (may be absent), turned q
    int64_t ys[3][2];
    int heads[3];
    uint8_t* cache[2];  // k, v
    uint8_t* par[2];    // 4 bits
    const int32_t* table;
    KvPlan plan;
    uint32_t* status;
    const double* freqs;  // null: no turn (rot == 0)
    int N, d, rot, n_pages, log_page, max_pages, inter;
    SmallDiv tile, per;
    float amp;
    uint64_t sig;
};

// A tile's tokens.
struct KvSlots {
    int seq[kRotMaxTile], slot[kRotMaxTile];  // slot: page << log_page | place, -1: none
};

__device__ __forceinline__ int64_t kv_cache_row(int slot, int log_page, int kv_heads, int h) {
    const int page = slot >> log_page;
    return (int64_t(int64_t(page) * kv_heads + h) << log_page) + (slot & ((1 << log_page) - 1));
}

// Four lanes (lane & 3 = cc) hold the 32 values of group gr of a row, eight
// each.  All lanes of the warp take part; `on`: this lane has values.
// A code is x' = (x - mid) / scale rounded: the quotient by the reciprocal is
// off by under 2^-19 (values of at most 8.1, three roundings), so only one
// that close to a border between codes is divided for.
__device__ __forceinline__ void quantise8(const float (&x)[8], bool is_k, bool on, int cc, int gr, int groups,
                                          uint8_t* codes, uint8_t* par, float& scale, float& mid, uint32_t& w) {
    float lo = x[0], hi = x[0], bad = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
        bad = fmaf(x[i], 0.f, bad);  // 0, or NaN for infinities and NaN
    }
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(~0u, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(~0u, hi, o));
        bad += __shfl_xor_sync(~0u, bad, o);
    }
    const __half hs = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f));
    scale = __half2float(hs);
    __half hm = __float2half_rn(__fadd_rn(lo, __fmul_rn(8.f, scale)));
    if (bad != bad) hm = __float2half_rn(bad);
    mid = __half2float(hm);
    const float inv = scale > 0.f ? __frcp_rn(scale) : 0.f;  // scale 0: all codes 8
    constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to a whole number, ties to even
    w = 0;
    bool near = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float q = fminf(fmaxf(__fmul_rn(__fsub_rn(x[i], mid), inv), -8.f), 7.f);
        const float r = __fadd_rn(q, kRound + 8.f);
        near |= fabsf(__fsub_rn(q, __fsub_rn(r, kRound + 8.f))) > 0.5f - 1.f / 262144.f;
        w |= (__float_as_uint(r) & 15u) << (4 * i);
    }
    if (near && scale > 0.f) {
        w = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = fminf(fmaxf(__fdiv_rn(__fsub_rn(x[i], mid), scale), -8.f), 7.f);
            w |= (__float_as_uint(__fadd_rn(q, kRound + 8.f)) & 15u) << (4 * i);
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

// grid: tiles of tokens.  smem: (cos, sin) [tile][rot/2]; 4 bits: the turned
// k and v rows [k heads + v heads][tile][d] in 16 bits.
template <typename T, int kBits, bool kVec>
__global__ void __launch_bounds__(kRotThreads) kv_append_kernel(const __grid_constant__ KvAppendParams p) {
    extern __shared__ __align__(16) uint8_t s_raw[];
    __shared__ KvSlots sl;
    if (p.plan.sig[0] != p.sig) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusBadPlan);
        return;
    }
    const int tile = p.tile.by, per = p.per.by;
    const int n0 = blockIdx.x * tile, nt = min(tile, p.N - n0), half = p.rot / 2;
    float2* s_cs = reinterpret_cast<float2*>(s_raw);
    T* s_row = reinterpret_cast<T*>(s_raw + ((size_t(tile) * half * 8 + 15) & ~size_t(15)));
    auto ready = [&] {
        if (threadIdx.x < nt) {
            const int t = threadIdx.x, seq = p.plan.row_seq[n0 + t], pos = p.plan.row_pos[n0 + t];
            int slot = -1;
            if (seq >= 0) {
                const int page = p.table[int64_t(seq) * p.max_pages + (pos >> p.log_page)];
                if (static_cast<unsigned>(page) < static_cast<unsigned>(p.n_pages))
                    slot = (page << p.log_page) + (pos & ((1 << p.log_page) - 1));
                else
                    atomicOr(p.status, kStatusBadCache);
            }
            sl.seq[t] = seq;
            sl.slot[t] = slot;
        }
        for (int i = threadIdx.x; i < nt * half; i += kRotThreads) {
            const int t = i / half, f = i - t * half;
            s_cs[i] = turn_of(p.plan.row_pos[n0 + t], p.freqs[f], p.amp, false);
        }
        __syncthreads();
    };
    const int kv = p.heads[0];
    // item or value i: a row (head of k, v or q, and token) and the place in it
    auto place = [&](int i, int& w, int& h, int& t, int& it) {
        const int row = p.per.div(i);
        it = i - row * per;
        h = p.tile.div(row);
        t = row - h * tile;
        w = h < kv ? 0 : h < 2 * kv ? 1 : 2;
        h -= w * kv;
    };
    auto from = [&](int w, int h, int t) {
        return static_cast<const T*>(p.x[w]) + (n0 + t) * p.xs[w][0] + h * p.xs[w][1];
    };
    // where a row goes: q to its dense row, k and v to the cache (or to shared memory, to be
    // quantised) and, if asked for, to a dense row too
    auto to = [&](int w, int h, int t, T*(&dst)[2]) {
        dst[0] = dst[1] = nullptr;
        if (w == 2) {
            dst[0] = static_cast<T*>(p.y[2]) + (n0 + t) * p.ys[2][0] + h * p.ys[2][1];
        } else if (kBits == 4) {
            dst[0] = s_row + (size_t(w * kv + h) * tile + t) * p.d;
        } else {
            if (sl.slot[t] >= 0)
                dst[0] = reinterpret_cast<T*>(p.cache[w]) + kv_cache_row(sl.slot[t], p.log_page, kv, h) * p.d;
            if (p.y[w]) dst[1] = static_cast<T*>(p.y[w]) + (n0 + t) * p.ys[w][0] + h * p.ys[w][1];
        }
    };
    const int n = (2 * kv + p.heads[2]) * tile * per;
    if constexpr (kVec) {
        move_items<T>(
            n,
            [&](int i, int& e0, int& e1) -> const T* {
                int w, h, t, it;
                place(i, w, h, t, it);
                item_at(it, w == 1 ? 0 : p.rot, p.inter, e0, e1);
                return t < nt ? from(w, h, t) : nullptr;
            },
            ready,
            [&](int i, int e0, int e1, float(&u)[8], float(&v)[8]) {
                int w, h, t, it;
                place(i, w, h, t, it);
                if (sl.seq[t] < 0) return;  // a row behind the last sequence stays as it was
                turn_item(u, v, e0, e1, w == 1 ? 0 : p.rot, p.inter, s_cs + t * half);
                T* dst[2];
                to(w, h, t, dst);
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (dst[k]) {
                        RowIo<T>::store8(dst[k] + e0, u);
                        RowIo<T>::store8(dst[k] + e1, v);
                    }
            });
    } else {
        ready();
        for (int i = threadIdx.x; i < n; i += kRotThreads) {
            int w, h, t, it;
            place(i, w, h, t, it);
            if (t >= nt || sl.seq[t] < 0) continue;
            const T* x = from(w, h, t);
            const float v = turn_one([&](int e) { return RowIo<T>::load(x + e); }, it, w == 1 ? 0 : p.rot, p.inter,
                                     s_cs + t * half);
            T* dst[2];
            to(w, h, t, dst);
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (dst[k]) RowIo<T>::store(dst[k] + it, v);
        }
    }
    if constexpr (kBits == 4) {
        __syncthreads();
        const int groups = p.d / 32, log_chunks = p.d == 64 ? 3 : 4;
        const int m = (2 * kv * tile) << log_chunks;  // a multiple of 8
        for (int i0 = 0; i0 < m; i0 += kRotThreads) {
            const int i = i0 + threadIdx.x, row = i >> log_chunks, ch = i & ((1 << log_chunks) - 1);
            const int hh = p.tile.div(row), t = row - hh * tile, w = hh < kv ? 0 : 1, h = hh - w * kv;
            const bool live = i < m && t < nt && sl.seq[t] >= 0;
            float u[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (live) RowIo<T>::widen(reinterpret_cast<const uint4*>(s_row + size_t(row) * p.d + 8 * ch), u);
            const bool on = live && sl.slot[t] >= 0;
            const int64_t r = on ? kv_cache_row(sl.slot[t], p.log_page, kv, h) : 0;
            float scale, mid;
            uint32_t codes;
            quantise8(u, w == 0, on, ch & 3, ch >> 2, groups, p.cache[w & 1] + r * (p.d / 2),
                      p.par[w & 1] + r * (4 * groups), scale, mid, codes);
            if (live && p.y[w]) {
                T* y = static_cast<T*>(p.y[w]) + (n0 + t) * p.ys[w][0] + h * p.ys[w][1] + 8 * ch;
#pragma unroll
                for (int k = 0; k < 8; ++k) u[k] = fmaf(scale, float((codes >> (4 * k)) & 15u) - 8.f, mid);
                if constexpr (kVec) RowIo<T>::store8(y, u);
                else
#pragma unroll
                    for (int k = 0; k < 8; ++k) RowIo<T>::store(y + k, u[k]);
            }
        }
    }
}

}  // namespace lf
