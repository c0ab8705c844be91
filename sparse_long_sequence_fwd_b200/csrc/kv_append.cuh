// kv_append.cuh -- a step's new tokens into the paged cache: the keys turned
// by their positions (rotary.cuh), the values as they are, both in 16 bits or
// quantised to 4; the queries turned beside them into dense rows, and, where
// the caller asks for them, the values that the cache now holds.
//
// 4 bits (groups of 32 values x of the row, in the 16-bit type):
//   scale = fp16((max - min) / 15), mid = fp16(min + 8 scale),
//   c = clamp(round((x - mid) / scale) + 8, 0, 15)   (ties to even; 8 if scale is 0)
// and the group stands for mid + scale (c - 8).  A group with an infinity or
// a NaN is held as NaN (mid).  The subtraction and the division are IEEE
// ones, so that the codes are the formula's also next to a border.
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
    int N, d, rot, tile, n_pages, log_page, max_pages, inter;
    float amp;
    uint64_t sig;
};

// The row of `cache` (in units of rows) for one token and kv head; -1: none.
struct KvSlots {
    int seq[kRotMaxTile], pos[kRotMaxTile], slot[kRotMaxTile];  // slot: page << log_page | place, -1: none
};

__device__ __forceinline__ int64_t kv_cache_row(int slot, int log_page, int kv_heads, int h) {
    const int page = slot >> log_page;
    return (int64_t(int64_t(page) * kv_heads + h) << log_page) + (slot & ((1 << log_page) - 1));
}

// Four lanes (lane & 3 = cc) hold the 32 values of group gr of a row, eight
// each.  All lanes of the warp take part; `on`: this lane has values.
template <bool kHalf>
__device__ __forceinline__ void quantise8(const float (&x)[8], bool is_k, bool on, int cc, int gr, int groups,
                                          uint8_t* codes, uint8_t* par, float (&held)[8]) {
    float lo = x[0], hi = x[0], bad = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
        bad += x[i] - x[i];  // 0, or NaN for infinities and NaN
    }
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(~0u, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(~0u, hi, o));
        bad += __shfl_xor_sync(~0u, bad, o);
    }
    const __half hs = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f));
    const float scale = __half2float(hs);
    __half hm = __float2half_rn(__fadd_rn(lo, __fmul_rn(8.f, scale)));
    if (bad != bad) hm = __float2half_rn(bad);
    const float mid = __half2float(hm);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float c = 8.f;
        if (scale > 0.f) c = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(x[i], mid), scale)) + 8.f, 0.f), 15.f);
        w |= static_cast<uint32_t>(c) << (4 * i);
        held[i] = mid + scale * (c - 8.f);
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
    constexpr bool kHalf = sizeof(T) == 2 && !std::is_same<T, __nv_bfloat16>::value;
    if (p.plan.sig[0] != p.sig) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusBadPlan);
        return;
    }
    const int n0 = blockIdx.x * p.tile, nt = min(p.tile, p.N - n0), half = p.rot / 2;
    float2* s_cs = reinterpret_cast<float2*>(s_raw);
    T* s_row = reinterpret_cast<T*>(s_raw + ((size_t(p.tile) * half * 8 + 15) & ~size_t(15)));
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
        sl.pos[t] = pos;
        sl.slot[t] = slot;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nt * half; i += kRotThreads) {
        const int t = i / half, f = i - t * half;
        s_cs[i] = turn_of(sl.pos[t], p.freqs[f], p.amp, false);
    }
    __syncthreads();
    const int kv = p.heads[0];
    const int heads = 2 * kv + p.heads[2];
    const int per = kVec ? p.d / 16 : p.d;
    const int n = heads * nt * per;
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kRotThreads) {
        const int row = i / per, it = i - row * per;
        int h = row / nt;
        const int hh = h, t = row - h * nt;
        const int w = h < kv ? 0 : h < 2 * kv ? 1 : 2;
        h -= w * kv;
        if (sl.seq[t] < 0) continue;  // a row behind the last sequence stays as it was
        const T* x = static_cast<const T*>(p.x[w]) + (n0 + t) * p.xs[w][0] + h * p.xs[w][1];
        const int rot = w == 1 ? 0 : p.rot;
        // where the row goes: q to its dense row, k and v to the cache (or to shared memory, to be
        // quantised) and, if asked for, to a dense row too
        T* dst[2] = {nullptr, nullptr};
        if (w == 2) {
            dst[0] = static_cast<T*>(p.y[2]) + (n0 + t) * p.ys[2][0] + h * p.ys[2][1];
        } else if (kBits == 4) {
            dst[0] = s_row + (size_t(hh) * nt + t) * p.d;
        } else {
            if (sl.slot[t] >= 0) dst[0] = reinterpret_cast<T*>(p.cache[w]) + kv_cache_row(sl.slot[t], p.log_page, kv, h) * p.d;
            if (p.y[w]) dst[1] = static_cast<T*>(p.y[w]) + (n0 + t) * p.ys[w][0] + h * p.ys[w][1];
        }
        if constexpr (kVec) {
            int e0, e1;
            item_at(it, rot, p.inter, e0, e1);
            float u[8], v[8];
            RowIo<T>::load8(x + e0, u);
            RowIo<T>::load8(x + e1, v);
            turn_item(u, v, e0, e1, rot, p.inter, s_cs + t * half);
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (dst[k]) {
                    RowIo<T>::store8(dst[k] + e0, u);
                    RowIo<T>::store8(dst[k] + e1, v);
                }
        } else {
            const float v = turn_one([&](int e) { return RowIo<T>::load(x + e); }, it, rot, p.inter, s_cs + t * half);
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (dst[k]) RowIo<T>::store(dst[k] + it, v);
        }
    }
    if constexpr (kBits == 4) {
        __syncthreads();
        const int chunks = p.d / 8, groups = p.d / 32;  // d is 64 or 128
        const int m = 2 * kv * nt * chunks;             // a multiple of 8
        for (int i0 = 0; i0 < m; i0 += kRotThreads) {
            const int i = i0 + threadIdx.x;
            const bool there = i < m;
            const int row = there ? i / chunks : 0, ch = there ? i - row * chunks : 0;
            const int hh = row / nt, t = row - hh * nt, w = hh < kv ? 0 : 1, h = hh - w * kv;
            const bool live = there && sl.seq[t] >= 0;
            float u[8], held[8];
            if (live) RowIo<T>::load8_shared(s_row + size_t(row) * p.d + 8 * ch, u);
            else
#pragma unroll
                for (int k = 0; k < 8; ++k) u[k] = 0.f;
            const bool on = live && sl.slot[t] >= 0;
            const int64_t r = on ? kv_cache_row(sl.slot[t], p.log_page, kv, h) : 0;
            quantise8<kHalf>(u, w == 0, on, ch & 3, ch >> 2, groups, p.cache[w] + r * (p.d / 2),
                             p.par[w] + r * (4 * groups), held);
            if (live && p.y[w]) {
                T* y = static_cast<T*>(p.y[w]) + (n0 + t) * p.ys[w][0] + h * p.ys[w][1];
                if constexpr (kVec) RowIo<T>::store8(y + 8 * ch, held);
                else
#pragma unroll
                    for (int k = 0; k < 8; ++k) RowIo<T>::store(y + 8 * ch + k, held[k]);
            }
        }
    }
}

}  // namespace lf
