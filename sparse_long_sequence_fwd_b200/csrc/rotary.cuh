// rotary.cuh -- rotary positions: dense rows (training, both directions) and
// new tokens on their way into the paged cache (serving).
//
// Pair i of a row's first `rot` values, (x, y), is turned by the angle
// t = position * freqs[i] and scaled by the amplitude a:
//   x' = a (x cos t - y sin t),  y' = a (y cos t + x sin t).
// The pairs are (i, i + rot/2), or (2i, 2i+1) when interleaved; the values
// behind rot are copied.  The gradient is the transpose, the turn by -t.
//
// Angles: position * freqs[i] is formed in 64 bits and reduced to a
// fraction of a turn there, because at position 10^6 a 32-bit angle is off
// by 2^-5 radians; what is left (within half a turn) is turned to 32 bits,
// where it is off by at most 2^-24 of half a turn, and sincospif takes it
// from there.  The products are in 32 bits and rounded once, on store.
//
// Bound: bytes.  A value is read once and written once against 3 flops, so
// the kernels are copies that must not be slowed down by the trigonometry or
// by addresses.  A CTA takes a few tokens over all heads.  A thread has one
// place in the rows of one token (16 values: two 8-value chunks that are
// turned against each other) and takes it in every so-many-th head, so its
// eight (cos, sin) are read once, and a head costs an address and two wide
// loads and stores.  Its first kRotItems heads' loads are under way while the
// CTA computes the sines (one per thread, for all heads), into shared memory
// in an order in which a warp's reads meet every bank once.  Rows that 16-value
// items do not divide (half pairs with rot not a multiple of 16, strides or
// addresses off 16 bytes) are taken in the same way by pairs, two at a time
// where rot / 2 is even and all is aligned: a thread has its pairs of a row, with
// their (cos, sin), in every so-many-th head.
#pragma once
#include "lf_common.cuh"
#include "ptx.cuh"

namespace lf {

constexpr int kRotThreads = 128;
constexpr int kRotMaxD = 256;
constexpr int kRotMaxTile = 16;   // tokens per CTA

// Heads whose 16 values a thread holds at once: 64 bytes of either type.  Few,
// so that an SM holds seven CTAs of 72 registers, which spill 8 to 68 bytes a
// thread.  Over sets of inputs larger than L2: 4096 tokens of 36 rows of 64,
// bf16, 8.9 us (six CTAs, which spill none to 8 bytes, 9.8), fp32 gradients of
// 8192 tokens 19.0 (22.4), 16383 tokens of 32 rows, f16, 29.0 (28.0); eight
// spill up to 120 bytes and took 11.2 us where seven took 8.3.
template <typename T>
constexpr int kRotItems = 4 / int(sizeof(T));
constexpr int kRotCtas = 7;

// Eight values as loaded (kU 16-byte words), widened, and stored.
template <typename T>
struct RowIo;
template <>
struct RowIo<float> {
    static constexpr int kU = 2;
    static __device__ __forceinline__ void widen(const uint4* a, float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v[4 * i] = __uint_as_float(a[i].x);
            v[4 * i + 1] = __uint_as_float(a[i].y);
            v[4 * i + 2] = __uint_as_float(a[i].z);
            v[4 * i + 3] = __uint_as_float(a[i].w);
        }
    }
    static __device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
    static __device__ __forceinline__ float load(const float* p) { return *p; }
    static __device__ __forceinline__ void store(float* p, float v) { *p = v; }
};
template <>
struct RowIo<__nv_bfloat16> {
    static constexpr int kU = 1;
    static __device__ __forceinline__ void widen(const uint4* a, float (&v)[8]) {
        const uint32_t w[4] = {a->x, a->y, a->z, a->w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // bf16 is the upper half of fp32
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                  pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
    static __device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
};
template <>
struct RowIo<__half> {
    static constexpr int kU = 1;
    static __device__ __forceinline__ void widen(const uint4* a, float (&v)[8]) {
        const uint32_t w[4] = {a->x, a->y, a->z, a->w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
    static __device__ __forceinline__ void store8(__half* p, const float (&v)[8]) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]),
                                                  pack_f16x2(v[4], v[5]), pack_f16x2(v[6], v[7]));
    }
    static __device__ __forceinline__ float load(const __half* p) { return __half2float(*p); }
    static __device__ __forceinline__ void store(__half* p, float v) { *p = __float2half_rn(v); }
};

// (a cos t, a sin t) of a position and one frequency (radians per position).
__device__ __forceinline__ float2 turn_of(int pos, double freq, float amp, bool back) {
    const double turns = static_cast<double>(pos) * (freq * 0.15915494309189533577);  // / (2 pi)
    const float half_turns = static_cast<float>(2.0 * (turns - rint(turns)));
    float s, c;
    sincospif(half_turns, &s, &c);
    return make_float2(amp * c, amp * (back ? -s : s));
}

__device__ __forceinline__ void turn_pair(float& x, float& y, float2 cs) {
    const float t = x * cs.x - y * cs.y;
    y = y * cs.x + x * cs.y;
    x = t;
}

// Item `it` of a row (d / 16 items of 16 values): the elements at which its
// two 8-value chunks start.  Half pairs: item it < rot/16 holds chunks it and
// it + rot/16, turned against each other; every other item, and every
// interleaved one, is 16 neighbouring values.
__device__ __forceinline__ void item_at(int it, int rot, bool inter, int& e0, int& e1) {
    const bool split = !inter && it < rot / 16;
    e0 = split ? 8 * it : 16 * it;
    e1 = split ? 8 * it + rot / 2 : 16 * it + 8;
}

// A token's (cos, sin) in shared memory: pair f is at cs_at(f, half).  An
// item's eight pairs 8 i .. 8 i + 7 are four 16-byte words, word j of all
// items beside each other, and the next token's are 64 bytes further into the
// banks (half a row of 128), so that the words j of two tokens' four items,
// which eight lanes read together, are in different banks.
__host__ __device__ constexpr int cs_items(int half) { return (half + 7) / 8; }
__host__ __device__ constexpr int cs_stride(int half) {  // float2 per token
    return 8 * cs_items(half) + ((8 * cs_items(half)) % 16 == 0 ? 8 : 0);
}
__device__ __forceinline__ int cs_at(int f, int half) { return 2 * (((f & 7) >> 1) * cs_items(half) + (f >> 3)) + (f & 1); }

// Turns item `it` of a row with its eight pairs' cs (unused where all of
// the item's values are copied).
__device__ __forceinline__ void turn_item(float (&a)[8], float (&b)[8], int it, int rot, bool inter,
                                          const float2 (&cs)[8]) {
    if (!inter) {
        if (16 * it < rot) {
#pragma unroll
            for (int i = 0; i < 8; ++i) turn_pair(a[i], b[i], cs[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (16 * it + 2 * i < rot) turn_pair(a[2 * i], a[2 * i + 1], cs[i]);
            if (16 * it + 2 * i + 8 < rot) turn_pair(b[2 * i], b[2 * i + 1], cs[4 + i]);
        }
    }
}

// A row by pairs, kW at a time: rot / 2 pairs that are turned, then the others,
// neighbours.  Item `it`'s kW first and kW second values; e1 < 0 where the
// row ends before the second ones.
__host__ __device__ constexpr int pair_items(int d, int rot, int kw) { return (rot / 2 + (d - rot + 1) / 2 + kw - 1) / kw; }
template <int kW>
__device__ __forceinline__ void pair_at(int it, int d, int rot, bool inter, int& e0, int& e1) {
    const bool split = !inter && kW * it < rot / 2;
    e0 = split ? kW * it : 2 * kW * it;
    e1 = split ? kW * it + rot / 2 : 2 * kW * it + kW < d ? 2 * kW * it + kW : -1;
}

// kW neighbouring values of a row.
template <typename T, int kW>
struct __align__(kW * sizeof(T)) Few {
    T v[kW];
};

// move_rows for pairs; some heads at a time (six: the case of turn_kind's comment 13 us, eight: 17).
template <typename T, int kW, typename Ready, typename Sink>
__device__ __forceinline__ void move_pairs(const T* x, int stride, int first, int step, int heads, int e0, int e1,
                                           Ready ready, Sink sink) {
    constexpr int kHeads = kW * sizeof(T) > 4 ? 4 : 6;
    using Word = Few<T, kW>;
    bool fresh = true;
    do {
        Word raw[kHeads][2];
#pragma unroll
        for (int a = 0; a < kHeads; ++a) {
            const int h = first + a * step;
            if (h < heads) {
                const T* row = x + int64_t(h) * stride;
                raw[a][0] = *reinterpret_cast<const Word*>(row + e0);
                raw[a][1] = *reinterpret_cast<const Word*>(row + (e1 < 0 ? e0 : e1));
            }
        }
        if (fresh) ready();
        fresh = false;
#pragma unroll
        for (int a = 0; a < kHeads; ++a) {
            const int h = first + a * step;
            if (h < heads) {
                float u[kW], v[kW];
#pragma unroll
                for (int i = 0; i < kW; ++i) {
                    u[i] = RowIo<T>::load(&raw[a][0].v[i]);
                    v[i] = RowIo<T>::load(&raw[a][1].v[i]);
                }
                sink(h, u, v);
            }
        }
        first += kHeads * step;
    } while (first < heads);
}
template <typename T, int kW>
__device__ __forceinline__ void store_few(T* at, const float (&u)[kW]) {
    Few<T, kW> w;
#pragma unroll
    for (int i = 0; i < kW; ++i) RowIo<T>::store(&w.v[i], u[i]);
    *reinterpret_cast<Few<T, kW>*>(at) = w;
}

// A thread's item (16 values at e0 and e1 of a row) of heads first, first +
// step, .. below `heads`; head h's row is at x + h * stride.  ready() runs
// when the first loads are under way, sink(h, u, v) takes the widened chunks.
template <typename T, typename Ready, typename Sink>
__device__ __forceinline__ void move_rows(const T* x, int stride, int first, int step, int heads, int e0, int e1,
                                          Ready ready, Sink sink) {
    constexpr int kItems = kRotItems<T>, kU = RowIo<T>::kU;
    bool fresh = true;
    do {
        uint4 raw[kItems][2][kU];
#pragma unroll
        for (int a = 0; a < kItems; ++a) {
            const int h = first + a * step;
            if (h < heads) {
                const T* row = x + int64_t(h) * stride;
#pragma unroll
                for (int w = 0; w < kU; ++w) {
                    raw[a][0][w] = __ldcs(reinterpret_cast<const uint4*>(row + e0) + w);
                    raw[a][1][w] = __ldcs(reinterpret_cast<const uint4*>(row + e1) + w);
                }
            }
        }
        if (fresh) ready();
        fresh = false;
#pragma unroll
        for (int a = 0; a < kItems; ++a) {
            const int h = first + a * step;
            if (h < heads) {
                float u[8], v[8];
                RowIo<T>::widen(raw[a][0], u);
                RowIo<T>::widen(raw[a][1], v);
                sink(h, u, v);
            }
        }
        first += kItems * step;
    } while (first < heads);
}

// The eight pairs of an item, from a token's row of the table.
__device__ __forceinline__ void load_cs(float2 (&cs)[8], const float2* row, int it, int half) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float4 c = *reinterpret_cast<const float4*>(row + 2 * (j * cs_items(half) + it));
        cs[2 * j] = make_float2(c.x, c.y);
        cs[2 * j + 1] = make_float2(c.z, c.w);
    }
}

// ------------------------------------------------------------ dense rows

struct RotaryParams {
    const void* x[3];  // q, k, v: logical [B, heads, T, d], strides in elements
    void* y[3];
    int64_t xb[3], yb[3];  // sample
    int xh[3], xt[3];      // head, token
    int yh[3], yt[3];
    int heads[3];      // 0: absent
    const int32_t* pos;  // [B][T] (stride pos_stride, 0: shared), or null: 0 .. T-1
    int64_t pos_stride;
    const double* freqs;
    int B, T, d, rot;
    int log_tile, per;  // tokens per CTA; items per row
    int inter, back;
    float amp;
};

// kW: 0: items of 16 values, else pairs, kW at a time.
// grid: (tiles of tokens, B, 1 or 3): with 3 a CTA takes q, k or v only, where
// tiles alone are too few to fill the GPU.
template <typename Tin, typename Tout, int kW>
__global__ void __launch_bounds__(kRotThreads, kRotCtas) rotary_kernel(const __grid_constant__ RotaryParams p) {
    extern __shared__ __align__(16) float2 s_cs[];  // [tile][cs_stride]
    const int b = blockIdx.y, tile = 1 << p.log_tile, t0 = blockIdx.x * tile;
    const int nt = min(tile, p.T - t0), half = p.rot / 2, stride = cs_stride(half);
    const int w0 = gridDim.z == 1 ? 0 : blockIdx.z, w1 = gridDim.z == 1 ? 3 : w0 + 1;
    auto ready = [&] {
        for (int i = threadIdx.x; w0 < 2 && i < nt * half; i += kRotThreads) {
            const int t = i / half, f = i - t * half;
            const int pos = p.pos ? p.pos[b * p.pos_stride + t0 + t] : t0 + t;
            s_cs[t * stride + cs_at(f, half)] = turn_of(pos, p.freqs[f], p.amp, p.back);
        }
        __syncthreads();
    };
    // thread i has item i % per of token i / per % tile, and every step-th head
    const int rest = threadIdx.x / p.per, t = rest & (tile - 1), group = rest >> p.log_tile, it = threadIdx.x - rest * p.per;
    const int step = (kRotThreads / p.per) >> p.log_tile;
    int e0, e1;
    bool fresh = true;
    if constexpr (kW == 0) {
        item_at(it, p.rot, p.inter, e0, e1);
        float2 cs[8];
#pragma unroll 1
        for (int w = w0; w < w1; ++w) {
            if (p.heads[w] == 0) continue;
            const Tin* x = static_cast<const Tin*>(p.x[w]) + b * p.xb[w] + int64_t(t0 + t) * p.xt[w];
            Tout* y = static_cast<Tout*>(p.y[w]) + b * p.yb[w] + int64_t(t0 + t) * p.yt[w];
            const int yh = p.yh[w];
            move_rows<Tin>(
                x, p.xh[w], group < step && t < nt ? group : p.heads[w], step, p.heads[w], e0, e1,
                [&] {
                    if (!fresh) return;
                    fresh = false;
                    ready();
                    if (16 * it < p.rot && t < nt) load_cs(cs, s_cs + t * stride, it, half);
                },
                [&](int h, float(&u)[8], float(&v)[8]) {
                    if (w < 2) turn_item(u, v, it, p.rot, p.inter, cs);  // v is copied
                    Tout* row = y + int64_t(h) * yh;
                    RowIo<Tout>::store8(row + e0, u);
                    RowIo<Tout>::store8(row + e1, v);
                });
        }
    } else {
        pair_at<kW>(it, p.d, p.rot, p.inter, e0, e1);
        const bool turned = kW * it < half;
        float2 cs[kW];
#pragma unroll 1
        for (int w = w0; w < w1; ++w) {
            if (p.heads[w] == 0) continue;
            const Tin* x = static_cast<const Tin*>(p.x[w]) + b * p.xb[w] + int64_t(t0 + t) * p.xt[w];
            Tout* y = static_cast<Tout*>(p.y[w]) + b * p.yb[w] + int64_t(t0 + t) * p.yt[w];
            const int yh = p.yh[w];
            move_pairs<Tin, kW>(
                x, p.xh[w], group < step && t < nt ? group : p.heads[w], step, p.heads[w], e0, e1,
                [&] {
                    if (!fresh) return;
                    fresh = false;
                    ready();
                    if (turned && t < nt)
#pragma unroll
                        for (int i = 0; i < kW; ++i) cs[i] = s_cs[t * stride + cs_at(kW * it + i, half)];
                },
                [&](int h, float(&u)[kW], float(&v)[kW]) {
                    if (w < 2 && turned)
#pragma unroll
                        for (int i = 0; i < kW; ++i) turn_pair(u[i], v[i], cs[i]);
                    Tout* row = y + int64_t(h) * yh;
                    store_few<Tout, kW>(row + e0, u);
                    if (e1 >= 0) store_few<Tout, kW>(row + e1, v);
                });
        }
    }
}

}  // namespace lf
