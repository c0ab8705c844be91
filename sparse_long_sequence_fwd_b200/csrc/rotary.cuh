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
// the kernels are copies that must not be slowed down by the trigonometry.
// A CTA takes a few tokens over all heads: the sines of a token are computed
// once into shared memory and serve its q and k heads (36 rows a token at
// 12 heads).  A thread moves items of 16 values (two 8-value chunks that are
// turned against each other); the loads of a CTA's first 1024 items (512 from
// fp32), which is all of them where a token has no more, are in flight before
// the sines are computed, so the two overlap.
#pragma once
#include "lf_common.cuh"
#include "ptx.cuh"

namespace lf {

constexpr int kRotThreads = 256;
constexpr int kRotMaxD = 256;
constexpr int kRotMaxTile = 16;   // tokens per CTA

// 16-value items that a thread holds at once: 128 bytes of either type.
template <typename T>
constexpr int kRotItems = 8 / int(sizeof(T));

// x / by for x < 2^20 and by <= 256: magic = ceil(2^32 / by), unused for 1.
struct SmallDiv {
    uint32_t by, magic;
    __device__ __forceinline__ int div(int x) const { return by == 1 ? x : int(__umulhi(uint32_t(x), magic)); }
};
inline SmallDiv small_div(int by) {
    return SmallDiv{uint32_t(by), by == 1 ? 0u : uint32_t((0x100000000ull + by - 1) / by)};
}

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

// Turns an item; cs: the token's rot/2 (cos, sin) in shared memory.
__device__ __forceinline__ void turn_item(float (&a)[8], float (&b)[8], int e0, int e1, int rot, bool inter,
                                          const float2* cs) {
    if (!inter) {
        if (e0 < rot) {
#pragma unroll
            for (int i = 0; i < 8; ++i) turn_pair(a[i], b[i], cs[e0 + i]);
        }
    } else {
        if (e0 < rot) {
#pragma unroll
            for (int i = 0; i < 4; ++i) turn_pair(a[2 * i], a[2 * i + 1], cs[e0 / 2 + i]);
        }
        if (e1 < rot) {
#pragma unroll
            for (int i = 0; i < 4; ++i) turn_pair(b[2 * i], b[2 * i + 1], cs[e1 / 2 + i]);
        }
    }
}

// Value e of a row whose value f is at(f), turned (the element-wise path:
// head dimensions, rot or strides that the 16-value items do not divide).
template <typename At>
__device__ __forceinline__ float turn_one(At at, int e, int rot, bool inter, const float2* cs) {
    const float x = at(e);
    if (e >= rot) return x;
    const int h = rot / 2;
    const bool first = inter ? !(e & 1) : e < h;
    const int i = inter ? e >> 1 : (first ? e : e - h);
    const float y = at(inter ? e ^ 1 : (first ? e + h : e - h));
    return first ? x * cs[i].x - y * cs[i].y : x * cs[i].x + y * cs[i].y;
}

// A CTA's items 0 .. n-1, a thread's share of kRotItems at a time: source(i,
// e0, e1) gives the row and the two chunks' places in it (null: no such
// item), sink(i, e0, e1, u, v) takes the widened chunks.  ready() runs once,
// when the first loads are under way.
template <typename T, typename Source, typename Ready, typename Sink>
__device__ __forceinline__ void move_items(int n, Source source, Ready ready, Sink sink) {
    constexpr int kItems = kRotItems<T>, kU = RowIo<T>::kU;
    for (int i0 = 0; i0 < n; i0 += kItems * kRotThreads) {
        uint4 raw[kItems][2][kU];
        int e0[kItems], e1[kItems];
        bool there[kItems];
#pragma unroll
        for (int a = 0; a < kItems; ++a) {
            const int i = i0 + a * kRotThreads + threadIdx.x;
            const T* x = i < n ? source(i, e0[a], e1[a]) : nullptr;
            there[a] = x != nullptr;
            if (there[a])
#pragma unroll
                for (int w = 0; w < kU; ++w) {
                    raw[a][0][w] = __ldcs(reinterpret_cast<const uint4*>(x + e0[a]) + w);
                    raw[a][1][w] = __ldcs(reinterpret_cast<const uint4*>(x + e1[a]) + w);
                }
        }
        if (i0 == 0) ready();
#pragma unroll
        for (int a = 0; a < kItems; ++a)
            if (there[a]) {
                float u[8], v[8];
                RowIo<T>::widen(raw[a][0], u);
                RowIo<T>::widen(raw[a][1], v);
                sink(i0 + a * kRotThreads + threadIdx.x, e0[a], e1[a], u, v);
            }
    }
}

// ------------------------------------------------------------ dense rows

struct RotaryParams {
    const void* x[3];  // q, k, v: logical [B, heads, T, d], strides in elements
    void* y[3];
    int64_t xs[3][3];  // (b, h, t)
    int64_t ys[3][3];
    int heads[3];      // 0: absent
    const int32_t* pos;  // [B][T] (stride pos_stride, 0: shared), or null: 0 .. T-1
    int64_t pos_stride;
    const double* freqs;
    int B, T, d, rot;
    SmallDiv tile, per;  // tokens per CTA; items (kVec) or values per row
    int inter, back;
    float amp;
};

// grid: (tiles of tokens, B)
template <typename Tin, typename Tout, bool kVec>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
    extern __shared__ float2 s_cs[];  // [tile][rot/2]
    const int b = blockIdx.y, tile = p.tile.by, per = p.per.by, t0 = blockIdx.x * tile;
    const int nt = min(tile, p.T - t0), half = p.rot / 2;
    auto ready = [&] {
        for (int i = threadIdx.x; i < nt * half; i += kRotThreads) {
            const int t = i / half, f = i - t * half;
            const int pos = p.pos ? p.pos[b * p.pos_stride + t0 + t] : t0 + t;
            s_cs[i] = turn_of(pos, p.freqs[f], p.amp, p.back);
        }
        __syncthreads();
    };
    // item or value i: a row (head of q, k or v, and token) and the place in it
    auto place = [&](int i, int& w, int& h, int& t, int& it) {
        const int row = p.per.div(i);
        it = i - row * per;
        h = p.tile.div(row);
        t = row - h * tile;
        w = 0;
        if (h >= p.heads[0]) {
            h -= p.heads[0];
            w = 1;
            if (h >= p.heads[1]) {
                h -= p.heads[1];
                w = 2;
            }
        }
    };
    auto from = [&](int w, int h, int t) {
        return static_cast<const Tin*>(p.x[w]) + b * p.xs[w][0] + h * p.xs[w][1] + (t0 + t) * p.xs[w][2];
    };
    auto to = [&](int w, int h, int t) {
        return static_cast<Tout*>(p.y[w]) + b * p.ys[w][0] + h * p.ys[w][1] + (t0 + t) * p.ys[w][2];
    };
    const int n = (p.heads[0] + p.heads[1] + p.heads[2]) * tile * per;
    if constexpr (kVec) {
        move_items<Tin>(
            n,
            [&](int i, int& e0, int& e1) -> const Tin* {
                int w, h, t, it;
                place(i, w, h, t, it);
                item_at(it, w == 2 ? 0 : p.rot, p.inter, e0, e1);
                return t < nt ? from(w, h, t) : nullptr;
            },
            ready,
            [&](int i, int e0, int e1, float(&u)[8], float(&v)[8]) {
                int w, h, t, it;
                place(i, w, h, t, it);
                turn_item(u, v, e0, e1, w == 2 ? 0 : p.rot, p.inter, s_cs + t * half);  // v is copied
                Tout* y = to(w, h, t);
                RowIo<Tout>::store8(y + e0, u);
                RowIo<Tout>::store8(y + e1, v);
            });
    } else {
        ready();
        for (int i = threadIdx.x; i < n; i += kRotThreads) {
            int w, h, t, it;
            place(i, w, h, t, it);
            if (t >= nt) continue;
            const Tin* x = from(w, h, t);
            RowIo<Tout>::store(to(w, h, t) + it, turn_one([&](int e) { return RowIo<Tin>::load(x + e); }, it,
                                                          w == 2 ? 0 : p.rot, p.inter, s_cs + t * half));
        }
    }
}

}  // namespace lf
