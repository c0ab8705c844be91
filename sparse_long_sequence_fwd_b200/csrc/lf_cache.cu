// lf_cache.cu -- host side of the rotary positions and of the paged cache:
// argument checks and launches.  No workspace is kept here: plan and partial
// states live in buffers of the caller, so calls on different streams only
// share the device's status word.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "lf_attn.h"
#include "kv_append.cuh"
#include "kv_attn.cuh"
#include "kv_plan.cuh"
#include "lf_common.cuh"
#include "lf_host.h"
#include "rotary.cuh"

namespace {

using namespace lf;

constexpr double kLog2e = 1.4426950408889634;
// The attention's CTAs: as many as a 148-SM B200 holds at once (larger GPUs run
// it on as many), so plan and workspace have sizes known without a device.
int kv_grid(int d, int bits, int rows, bool pack) { return 148 * kv_ctas_per_sm(d, bits, rows > 8, pack); }
static_assert(148 * 4 <= kKvMaxCtas, "");
constexpr int kMaxRotHeads = 1024;
constexpr int kAppendSmem = 100 * 1024;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t size_of(lf_dtype t) { return t == LF_F32 ? 4 : 2; }
bool known(lf_dtype t) { return t == LF_F32 || t == LF_BF16 || t == LF_F16; }

// The bytes that a strided tensor reaches over.
struct Span {
    uintptr_t lo = 0, hi = 0;
    bool meets(const Span& o) const { return lo < o.hi && o.lo < hi; }
};

// The strides that are stepped by: nothing steps along a dimension of one, whatever its stride.
template <int kDims>
struct Strides {
    int64_t s[kDims];
    Strides(const int64_t* n, const int64_t* given) {
        for (int i = 0; i < kDims; ++i) s[i] = n[i] > 1 ? given[i] : 0;
    }
};

// Sizes n[i] with strides s[i] (elements) and d contiguous values behind.
// False: a negative stride, or a place past 2^46 bytes.
bool span_of(const void* p, int dims, const int64_t* n, const int64_t* s, int d, size_t es, Span* out) {
    uint64_t last = 0;
    for (int i = 0; i < dims; ++i) {
        if (s[i] < 0) return false;
        if (n[i] <= 1 || s[i] == 0) continue;
        if (uint64_t(s[i]) > (uint64_t(1) << 44) / uint64_t(n[i])) return false;
        last += uint64_t(n[i] - 1) * uint64_t(s[i]);
    }
    if (last > (uint64_t(1) << 44)) return false;
    out->lo = reinterpret_cast<uintptr_t>(p);
    out->hi = out->lo + (last + uint64_t(d)) * es;
    return true;
}

// Rows that are written must not lie on one another.  False where two that differ along one dimension or two certainly do.
bool distinct(int dims, const int64_t* n, const int64_t* s, int d) {
    for (int i = 0; i < dims; ++i) {
        if (n[i] > 1 && s[i] < d) return false;
        for (int j = 0; j < i; ++j) {
            if (n[i] <= 1 || n[j] <= 1) continue;
            const int a = s[i] >= s[j] ? i : j, b = i + j - a;  // a has the larger stride
            if (s[a] >= (n[b] - 1) * s[b] + d) continue;
            for (int64_t k = 1; k < std::min<int64_t>(n[b], 4096); ++k) {  // k steps along b against the nearest along a
                const int64_t m = k * s[b] / s[a], rest = k * s[b] - m * s[a];
                if ((m < n[a] && rest < d) || (m + 1 < n[a] && s[a] - rest < d)) return false;
            }
        }
    }
    return true;
}
bool same_twice(const void* const* p, int n) {
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < i; ++j)
            if (p[i] && p[i] == p[j]) return true;
    return false;
}

bool by_eight(const void* p, int dims, const int64_t* s, size_t es) {
    if (!aligned(p, 16)) return false;
    for (int i = 0; i < dims; ++i)
        if ((s[i] * int64_t(es)) % 16 != 0) return false;
    return true;
}

// Tokens per CTA (a power of two): as many as leave a thread about five heads'
// 16 values, so that the sines are few beside them, and no fewer CTAs than
// two per SM.  (4096 tokens of 36 rows of 64: 4 tokens, 1024 CTAs; half or
// twice as many heads a thread took 10.5 and 10.6 us against 8.5.)
// Where 4-bit rows follow through shared memory, twice as many heads (16384
// tokens of 32 rows: 47 -> 44 us).
int log_tile_for(int64_t tokens, int heads, int d, int per, bool staged) {
    int n = 0;
    while ((2 << n) <= kRotMaxTile && (2 << n) * per <= kRotThreads &&
           int64_t(2 << n) * d * heads <= int64_t(kRotThreads) * (staged ? 160 : 80) && tokens >= int64_t(2 << n) * 296)
        ++n;
    return n;
}

// CTAs for q, k and v apart, where tiles of one token are under two per SM.
int apart(int64_t tiles) { return tiles < 296 ? 3 : 1; }

bool small(const int64_t* s) { return s[0] <= INT32_MAX && s[1] <= INT32_MAX; }

template <typename Tin, typename Tout>
void launch_rotary(const RotaryParams& p, int kw, dim3 grid, size_t smem, cudaStream_t s) {
    if (kw == 0) rotary_kernel<Tin, Tout, 0><<<grid, kRotThreads, smem, s>>>(p);
    else if (kw == 1) rotary_kernel<Tin, Tout, 1><<<grid, kRotThreads, smem, s>>>(p);
    else rotary_kernel<Tin, Tout, 2><<<grid, kRotThreads, smem, s>>>(p);
}

// How rows are taken: 0: by items of 16 values, else by pairs, so many at a time.  wide: rows begin at 16-byte
// boundaries.  (4099 tokens, 36 rows of 64, 24 of them turned, half pairs: 13 us by
// two, 17 by one; 45 value by value.)
int turn_kind(bool wide, int d, int rot, bool inter) {
    if (wide && d % 16 == 0 && (inter || rot % 16 == 0)) return 0;
    return wide && !inter && rot % 4 == 0 && d % 2 == 0 ? 2 : 1;
}

uint64_t mix(uint64_t h, uint64_t x) {  // a 64-bit value at a time, upper halves folded back
    h = (h ^ x) * 0x9e3779b97f4a7c15ull;
    return h ^ (h >> 32);
}

int heads_of_unit(int group, int nsub) { return (group + nsub - 1) / nsub; }
int unit_rows(const KvShape& sh) { return heads_of_unit(sh.q_heads / sh.kv_heads, sh.nsub) * sh.tpt; }

// Whether units (of up to `keys` keys) are cut between the CTAs.  Whole, the
// CTAs take ceil(units / grid) rounds of them; cut, units / grid, and a merge
// that costs about as much as kCutKeys keys (one token, 12 heads, 258 keys:
// 6.2 us whole, 8.4 cut; 24 tokens, 2 heads, 1029 keys: 30 whole, 17 cut).
// Long ones are always cut, since their lengths may differ.
constexpr int64_t kCutKeys = 320, kLongKeys = 4096;
bool cut_units(int64_t units, int64_t keys, int64_t grid) {
    const int64_t rounds = (units + grid - 1) / grid;
    return keys > kLongKeys || keys * (rounds * grid - units) > kCutKeys * grid;
}
// Tiles are cut for a short last round only where there are few rounds, counted
// as if every tile were full, so that a workspace's size need not know the
// sequences: whether tiles of so many rows may be cut at all.
constexpr int64_t kTileRounds = 4;
bool may_cut_tiles(int64_t rows, int tpt, int kv_heads, int64_t keys, int64_t grid) {
    return keys > kLongKeys || (keys > kCutKeys && (rows + tpt - 1) / tpt * kv_heads < kTileRounds * grid);
}

// Rows of a tile: as many as the sequences have each, up to what a unit holds.
// Times in us, tiles against single rows: 4096 rows of a prompt, 12 heads of 64,
// window 256: 71 : 481 (4 bits 84 : 579); 16 sequences of 4 drafts, 4000 keys,
// 32 heads on 8 of 128: 53 : 148 (4 bits 63 : 97).
// No tiles where heads are dilated, whose neighbouring rows share no keys.  Not
// two rows in a unit of 16 either, which costs what two units of 8 do (8
// sequences of 3, 8000 keys, 16 heads on 2 of 128: 32 against 28).
int tile_of(const KvShape& sh, int d, int bits) {
    const int group = sh.q_heads / sh.kv_heads;
    if (!sh.one_dil || sh.dil[0] != 1 || sh.N < 2 * int64_t(sh.S)) return 1;
    const int t = static_cast<int>(std::min<int64_t>(kv_tile_rows(d, bits) / group, (int64_t(sh.N) + sh.S - 1) / sh.S));
    return std::max(1, t * group > 8 && t < 3 ? 8 / group : t);
}

// How work of tiles of up to tpt rows is split.
void split_work(KvShape* sh, int d, int bits, int tpt) {
    sh->tpt = tpt;
    const int64_t keys = std::min<int64_t>(int64_t(sh->r) + tpt, sh->max_len) + sh->n_global;
    const int64_t tiles = tpt > 1 ? std::min(sh->N, sh->N / tpt + sh->S) : sh->N;
    const int64_t blocks = (keys + sh->block - 1) / sh->block, units = tiles * sh->kv_heads * sh->nsub;
    const int64_t grid = kv_grid(d, bits, unit_rows(*sh), tpt > 1);
    sh->may_cut = tpt == 1 || may_cut_tiles(sh->N, tpt, sh->kv_heads, keys, grid);
    sh->cut = sh->may_cut && cut_units(units, keys, grid);
    // no more CTAs than blocks that ordinary rows can have
    sh->G = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(grid, blocks * std::min(units, grid))));
}

lf_status kv_shape(int S, int N, int n_global, int page, int max_pages, int q_heads, int kv_heads, int d, int bits,
                   int r, const int32_t* dil, KvShape* sh) {
    if (S < 1 || N < 0 || n_global < 0 || page < 1 || max_pages < 1 || q_heads < 1 || kv_heads < 1 || r < 0)
        return LF_ERR_INVALID_ARG;
    if (q_heads % kv_heads != 0 || d < 1 || (bits != 16 && bits != 4)) return LF_ERR_INVALID_ARG;
    if (dil)
        for (int h = 0; h < kv_heads && h < kMaxHeads; ++h)
            if (dil[h] < 1) return LF_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return LF_ERR_UNSUPPORTED;
    if (page < 8 || page > 256 || (page & (page - 1)) != 0) return LF_ERR_UNSUPPORTED;
    if (q_heads > kMaxHeads || n_global > kKvMaxGlobal || S > (1 << 20) || N > (1 << 20)) return LF_ERR_UNSUPPORTED;
    if (int64_t(max_pages) * page > (int64_t(1) << 30)) return LF_ERR_UNSUPPORTED;
    if (int64_t(S) * std::max(n_global, max_pages) > (int64_t(1) << 40)) return LF_ERR_UNSUPPORTED;
    std::memset(sh, 0, sizeof(*sh));
    sh->S = S;
    sh->N = N;
    sh->n_global = n_global;
    sh->max_len = max_pages * page;
    sh->q_heads = q_heads;
    sh->kv_heads = kv_heads;
    const int group = q_heads / kv_heads;
    sh->nsub = (group + 15) / 16;
    sh->r = std::min(r, sh->max_len);
    sh->one_dil = 1;
    for (int h = 0; h < kv_heads; ++h) {
        sh->dil[h] = dil ? std::min(dil[h], sh->max_len) : 1;
        if (sh->dil[h] != sh->dil[0]) sh->one_dil = 0;
    }
    sh->block = kv_block(bits);
    split_work(sh, d, bits, 1);
    const int tpt = tile_of(*sh, d, bits);
    // (whole units of single rows that the CTAs hold at once: tiles are longer; 16 sequences of 2 rows, 12 heads of 64,
    // window 256: 9.4 us against 8.4)
    if (tpt > 1 && (sh->cut || int64_t(N) * kv_heads > kv_grid(d, bits, group, false))) split_work(sh, d, bits, tpt);
    uint64_t h = 14695981039346656037ull;
    for (int64_t x : {int64_t(S), int64_t(N), int64_t(page), int64_t(max_pages)}) h = mix(h, uint64_t(x));
    sh->sig_rows = h;
    for (int64_t x : {int64_t(n_global), int64_t(q_heads), int64_t(kv_heads), int64_t(sh->r), int64_t(d), int64_t(bits),
                      int64_t(sh->tpt)}) h = mix(h, uint64_t(x));
    for (int a = 0; a < kv_heads; ++a) h = mix(h, uint64_t(sh->dil[a]));
    sh->sig_all = h;
    return LF_OK;
}

uint64_t workspace_of(const KvShape& sh, int d, int bits) {
    const int rows = unit_rows(sh);
    return sh.cut ? uint64_t(2) * kv_grid(d, bits, rows, sh.tpt > 1) * rows * kv_piece_row(d) * sizeof(float) : 0;
}

int log2_of(int x) {
    int n = 0;
    while ((1 << n) < x) ++n;
    return n;
}

lf_status check_cache(const void* k, const void* v, const void* k_par, const void* v_par, int n_pages, int kv_heads,
                      int page, lf_dtype dtype, int bits) {
    if (!k || !v || n_pages < 1) return LF_ERR_INVALID_ARG;
    if ((bits == 4) != (k_par != nullptr) || (bits == 4) != (v_par != nullptr)) return LF_ERR_INVALID_ARG;
    for (const void* p : {k, v, k_par, v_par})
        if (!aligned(p, 16)) return LF_ERR_INVALID_ARG;
    if (!known(dtype)) return LF_ERR_INVALID_ARG;
    if (dtype == LF_F32) return LF_ERR_UNSUPPORTED;
    if (int64_t(n_pages) * kv_heads * page > INT32_MAX) return LF_ERR_UNSUPPORTED;
    return LF_OK;
}

using AttnKernel = void (*)(KvAttnParams);

template <int HD, int kBits>
AttnKernel attn_kernel(bool half, int unit_rows, bool pack, int* smem) {
    *smem = kv_attn_smem<HD, kBits>(unit_rows);
    if (pack) {
        if constexpr (kv_tile_rows(HD, kBits) > 8)
            if (unit_rows > 8) return half ? kv_attn_kernel<HD, kBits, true, 2, true> : kv_attn_kernel<HD, kBits, false, 2, true>;
        return half ? kv_attn_kernel<HD, kBits, true, 1, true> : kv_attn_kernel<HD, kBits, false, 1, true>;
    }
    if (unit_rows <= 8) return half ? kv_attn_kernel<HD, kBits, true, 1, false> : kv_attn_kernel<HD, kBits, false, 1, false>;
    return half ? kv_attn_kernel<HD, kBits, true, 2, false> : kv_attn_kernel<HD, kBits, false, 2, false>;
}

using AppendKernel = void (*)(KvAppendParams);

template <typename T, int kBits>
AppendKernel append_kernel(int kw) {
    return kw == 0 ? kv_append_kernel<T, kBits, 0> : kw == 1 ? kv_append_kernel<T, kBits, 1> : kv_append_kernel<T, kBits, 2>;
}

// Shared-memory limits of the kernels, once per device.
lf_status kernel_limits() {
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return LF_ERR_CUDA;
    std::lock_guard<std::mutex> lock(mu);
    if (done[dev]) return LF_OK;
    for (int half = 0; half < 2; ++half)
        for (int kind = 0; kind < 4; ++kind) {
            const int rows = kind & 1 ? 16 : 8;
            const bool pack = kind & 2;
            int smem[4];
            const AttnKernel kern[4] = {
                attn_kernel<64, 16>(half, rows, pack, &smem[0]), attn_kernel<64, 4>(half, rows, pack, &smem[1]),
                attn_kernel<128, 16>(half, rows, pack, &smem[2]), attn_kernel<128, 4>(half, rows, pack, &smem[3])};
            for (int a = 0; a < 4; ++a)
                if (cudaFuncSetAttribute(kern[a], cudaFuncAttributeMaxDynamicSharedMemorySize, smem[a]) != cudaSuccess ||
                    cudaFuncSetAttribute(kern[a], cudaFuncAttributePreferredSharedMemoryCarveout,
                                         cudaSharedmemCarveoutMaxShared) != cudaSuccess)
                    return LF_ERR_CUDA;
        }
    for (int kw = 0; kw < 3; ++kw)
        for (const AppendKernel kern : {append_kernel<__half, 4>(kw), append_kernel<__nv_bfloat16, 4>(kw)})
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kAppendSmem) != cudaSuccess)
                return LF_ERR_CUDA;
    done[dev] = true;
    return LF_OK;
}

}  // namespace

extern "C" {

lf_status lf_attn_rotary(const void* q, const void* k, const void* v, void* q_out, void* k_out, void* v_out,
                         const int64_t* strides, int B, int q_heads, int kv_heads, int T, int d, const int32_t* pos,
                         int64_t pos_stride, const double* freqs, int rot, int interleaved, int inverse,
                         float amplitude, lf_dtype in_dtype, lf_dtype out_dtype, void* stream) {
    const void* x[3] = {q, k, v};
    void* y[3] = {q_out, k_out, v_out};
    if (!strides || B < 0 || T < 0 || q_heads < 0 || kv_heads < 0 || d < 1 || rot < 0 || rot > d || (rot & 1) ||
        pos_stride < 0 || !std::isfinite(amplitude) || !known(in_dtype) || !known(out_dtype))
        return LF_ERR_INVALID_ARG;
    if ((rot > 0 && !freqs) || !aligned(freqs, 8) || !aligned(pos, 4)) return LF_ERR_INVALID_ARG;
    if (!q && !k && !v) return LF_ERR_INVALID_ARG;
    const size_t ei = size_of(in_dtype), eo = size_of(out_dtype);
    RotaryParams p{};
    Span in[3], out[3];
    bool wide = true, apart_rows = !same_twice(y, 3);
    for (int a = 0; a < 3; ++a) {
        if ((x[a] == nullptr) != (y[a] == nullptr)) return LF_ERR_INVALID_ARG;
        p.heads[a] = x[a] ? (a == 0 ? q_heads : kv_heads) : 0;
        if (!x[a]) continue;
        if (!aligned(x[a], ei) || !aligned(y[a], eo)) return LF_ERR_INVALID_ARG;
        const int64_t n[3] = {B, p.heads[a], T};
        const Strides<3> by_x(n, strides + 3 * a), by_y(n, strides + 9 + 3 * a);
        const int64_t *xs = by_x.s, *ys = by_y.s;
        if (!span_of(x[a], 3, n, xs, d, ei, &in[a]) || !span_of(y[a], 3, n, ys, d, eo, &out[a]))
            return LF_ERR_INVALID_ARG;
        apart_rows = apart_rows && distinct(3, n, ys, d);
        wide = wide && by_eight(x[a], 3, xs, ei) && by_eight(y[a], 3, ys, eo);
        p.x[a] = x[a];
        p.y[a] = y[a];
        if (!small(xs + 1) || !small(ys + 1)) return LF_ERR_UNSUPPORTED;
        p.xb[a] = xs[0];
        p.yb[a] = ys[0];
        p.xh[a] = static_cast<int>(xs[1]);
        p.yh[a] = static_cast<int>(ys[1]);
        p.xt[a] = static_cast<int>(xs[2]);
        p.yt[a] = static_cast<int>(ys[2]);
    }
    for (const Span& a : in)
        for (const Span& b : out)
            if (a.meets(b)) return LF_ERR_INVALID_ARG;
    if (in_dtype != out_dtype && in_dtype != LF_F32) return LF_ERR_UNSUPPORTED;
    if (d > kRotMaxD || q_heads > kMaxRotHeads || kv_heads > kMaxRotHeads || B > 65535) return LF_ERR_UNSUPPORTED;
    if (!apart_rows) return LF_ERR_INVALID_ARG;
    const int heads = p.heads[0] + p.heads[1] + p.heads[2];
    if (B == 0 || T == 0 || heads == 0) return LF_OK;
    p.pos = pos;
    p.pos_stride = pos_stride;
    p.freqs = freqs;
    p.B = B;
    p.T = T;
    p.d = d;
    p.rot = rot;
    p.inter = interleaved ? 1 : 0;
    p.back = inverse ? 1 : 0;
    p.amp = amplitude;
    const int kw = turn_kind(wide, d, rot, interleaved != 0);
    p.per = kw == 0 ? d / 16 : pair_items(d, rot, kw);
    p.log_tile = log_tile_for(int64_t(B) * T, heads, d, p.per, false);
    const unsigned tiles = (T + (1 << p.log_tile) - 1) >> p.log_tile;
    const dim3 grid(tiles, B, apart(int64_t(tiles) * B));
    const size_t smem = (size_t(cs_stride(rot / 2)) << p.log_tile) * sizeof(float2);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (in_dtype == LF_F32 && out_dtype == LF_F32) launch_rotary<float, float>(p, kw, grid, smem, s);
    else if (in_dtype == LF_F32 && out_dtype == LF_BF16) launch_rotary<float, __nv_bfloat16>(p, kw, grid, smem, s);
    else if (in_dtype == LF_F32) launch_rotary<float, __half>(p, kw, grid, smem, s);
    else if (in_dtype == LF_BF16) launch_rotary<__nv_bfloat16, __nv_bfloat16>(p, kw, grid, smem, s);
    else launch_rotary<__half, __half>(p, kw, grid, smem, s);
    return cudaGetLastError() == cudaSuccess ? LF_OK : LF_ERR_CUDA;
}

uint64_t lf_attn_cache_plan_bytes(int n_seqs, int n_tokens, int n_global) {
    if (n_seqs < 1 || n_tokens < 0 || n_global < 0 || n_seqs > (1 << 20) || n_tokens > (1 << 20) ||
        n_global > kKvMaxGlobal)
        return 0;
    return kv_plan_layout(n_seqs, n_tokens, n_global).total;
}

lf_status lf_attn_cache_plan(const int32_t* cu_tokens, const int32_t* context, int n_seqs, int n_tokens,
                             const int32_t* global_idx, int n_global, int page, int max_pages, int q_heads,
                             int kv_heads, int d, int bits, int r, const int32_t* dil, void* plan, void* stream) {
    if (!cu_tokens || !context || !plan || (n_global > 0) != (global_idx != nullptr)) return LF_ERR_INVALID_ARG;
    if (!aligned(cu_tokens, 4) || !aligned(context, 4) || !aligned(global_idx, 4) || !aligned(plan, 256))
        return LF_ERR_INVALID_ARG;
    KvShape sh;
    lf_status st = kv_shape(n_seqs, n_tokens, n_global, page, max_pages, q_heads, kv_heads, d, bits, r, dil, &sh);
    if (st != LF_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint32_t* status = nullptr;
    int sms = 0;
    if ((st = device_info(s, &status, &sms)) != LF_OK) return st;
    const KvPlan p = kv_plan_view(plan, kv_plan_layout(n_seqs, n_tokens, n_global));
    if (n_global > 0)
        kv_plan_globals_kernel<<<n_seqs, 256, 2 * sizeof(int32_t) * n_global, s>>>(global_idx, n_global, sh.max_len, p,
                                                                                 status);
    kv_plan_rows_kernel<<<1, kPlanThreads, 0, s>>>(cu_tokens, context, sh, p, status);
    return cudaGetLastError() == cudaSuccess ? LF_OK : LF_ERR_CUDA;
}

lf_status lf_attn_cache_append(const void* k, const void* v, const void* q, void* k_held, void* v_held, void* q_out,
                               const int64_t* strides, void* k_cache, void* v_cache, void* k_par, void* v_par,
                               int n_pages, int page, const int32_t* table, int max_pages, const void* plan, int n_seqs,
                               int n_tokens, int n_global, int q_heads, int kv_heads, int d, const double* freqs,
                               int rot, int interleaved, float amplitude, lf_dtype dtype, int bits, void* stream) {
    if (!k || !v || !strides || !table || !plan || (q != nullptr) != (q_out != nullptr)) return LF_ERR_INVALID_ARG;
    if (rot < 0 || rot > d || (rot & 1) || (rot > 0 && !freqs) || !aligned(freqs, 8) || !aligned(table, 4) ||
        !aligned(plan, 256) || !std::isfinite(amplitude))
        return LF_ERR_INVALID_ARG;
    KvShape sh;
    lf_status st = kv_shape(n_seqs, n_tokens, n_global, page, max_pages, q_heads, kv_heads, d, bits, 0, nullptr, &sh);
    if (st != LF_OK) return st;
    if ((st = check_cache(k_cache, v_cache, k_par, v_par, n_pages, kv_heads, page, dtype, bits)) != LF_OK) return st;
    KvAppendParams p{};
    const void* x[3] = {k, v, q};
    void* y[3] = {k_held, v_held, q_out};
    Span in[3], out[3];
    bool wide = true;
    for (int a = 0; a < 3; ++a) {
        p.heads[a] = a < 2 ? kv_heads : (q ? q_heads : 0);
        const int64_t n[2] = {n_tokens, p.heads[a]};
        const Strides<2> by_x(n, strides + 2 * a), by_y(n, strides + 6 + 2 * a);
        const int64_t *xs = by_x.s, *ys = by_y.s;
        if (x[a]) {
            if (!aligned(x[a], 2) || !span_of(x[a], 2, n, xs, d, 2, &in[a])) return LF_ERR_INVALID_ARG;
            if (!small(xs)) return LF_ERR_UNSUPPORTED;
            p.xt[a] = static_cast<int>(xs[0]);
            p.xh[a] = static_cast<int>(xs[1]);
            wide = wide && by_eight(x[a], 2, xs, 2);
        }
        if (y[a]) {
            if (!aligned(y[a], 2) || !span_of(y[a], 2, n, ys, d, 2, &out[a]) || !distinct(2, n, ys, d))
                return LF_ERR_INVALID_ARG;
            if (!small(ys)) return LF_ERR_UNSUPPORTED;
            p.yt[a] = static_cast<int>(ys[0]);
            p.yh[a] = static_cast<int>(ys[1]);
            wide = wide && by_eight(y[a], 2, ys, 2);
        }
        p.x[a] = x[a];
        p.y[a] = y[a];
    }
    for (const Span& a : in)
        for (const Span& b : out)
            if (a.meets(b)) return LF_ERR_INVALID_ARG;
    const void* const written[7] = {k_cache, v_cache, k_par, v_par, k_held, v_held, q_out};
    if (same_twice(written, 7)) return LF_ERR_INVALID_ARG;
    if (n_tokens == 0) return LF_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int sms = 0;
    if ((st = device_info(s, &p.status, &sms)) != LF_OK || (st = kernel_limits()) != LF_OK) return st;
    p.cache[0] = static_cast<uint8_t*>(k_cache);
    p.cache[1] = static_cast<uint8_t*>(v_cache);
    p.par[0] = static_cast<uint8_t*>(k_par);
    p.par[1] = static_cast<uint8_t*>(v_par);
    p.table = table;
    p.plan = kv_plan_view(const_cast<void*>(plan), kv_plan_layout(n_seqs, n_tokens, n_global));
    p.freqs = freqs;
    p.N = n_tokens;
    p.d = d;
    p.rot = rot;
    p.n_pages = n_pages;
    p.log_page = log2_of(page);
    p.max_pages = max_pages;
    p.inter = interleaved ? 1 : 0;
    p.amp = amplitude;
    p.sig = sh.sig_rows;
    const int kw = turn_kind(wide, d, rot, interleaved != 0);
    p.per = kw == 0 ? d / 16 : pair_items(d, rot, kw);
    p.log_tile = log_tile_for(n_tokens, 2 * kv_heads + p.heads[2], d, p.per, bits == 4);
    const size_t staged = bits == 4 ? size_t(2) * kv_heads * d * 2 : 0;  // per token
    const size_t smem = (size_t(cs_stride(rot / 2)) * sizeof(float2) + staged) << p.log_tile;
    const unsigned tiles = (n_tokens + (1 << p.log_tile) - 1) >> p.log_tile;
    const dim3 grid(tiles, apart(tiles));
    p.wide = wide ? 1 : 0;
    const AppendKernel kern = dtype == LF_F16 ? (bits == 16 ? append_kernel<__half, 16>(kw) : append_kernel<__half, 4>(kw))
                                              : (bits == 16 ? append_kernel<__nv_bfloat16, 16>(kw)
                                                            : append_kernel<__nv_bfloat16, 4>(kw));
    kern<<<grid, kRotThreads, smem, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? LF_OK : LF_ERR_CUDA;
}

uint64_t lf_attn_cache_workspace_bytes(int n_tokens, int n_global, int page, int max_pages, int q_heads, int kv_heads, int d,
                                       int bits, int r) {
    KvShape sh;
    // the most over all numbers of sequences and dilations
    if (kv_shape(1, n_tokens, n_global, page, max_pages, q_heads, kv_heads, d, bits, r, nullptr, &sh) != LF_OK) return 0;
    const int most = n_tokens < 2 ? 1 : std::max(1, 16 / (q_heads / kv_heads));
    uint64_t size = 0;
    for (int t = 1; t <= most; ++t) {
        split_work(&sh, d, bits, t);
        if (t > 1) sh.cut = sh.may_cut;
        size = std::max(size, workspace_of(sh, d, bits));
    }
    return size;
}

lf_status lf_attn_cache_fwd(const void* q, void* out, const int64_t* strides, const void* k_cache, const void* v_cache,
                            const void* k_par, const void* v_par, int n_pages, int page, const int32_t* table,
                            int max_pages, const void* plan, int n_seqs, int n_tokens, int n_global, int q_heads,
                            int kv_heads, int d, int r, const int32_t* dil, float scale, lf_dtype dtype, int bits,
                            void* workspace, uint64_t workspace_bytes, void* stream) {
    if (!q || !out || !strides || !table || !plan || !std::isfinite(scale)) return LF_ERR_INVALID_ARG;
    if (!aligned(table, 4) || !aligned(plan, 256) || !aligned(workspace, 16)) return LF_ERR_INVALID_ARG;
    KvShape sh;
    lf_status st = kv_shape(n_seqs, n_tokens, n_global, page, max_pages, q_heads, kv_heads, d, bits, r, dil, &sh);
    if (st != LF_OK) return st;
    if ((st = check_cache(k_cache, v_cache, k_par, v_par, n_pages, kv_heads, page, dtype, bits)) != LF_OK) return st;
    const int64_t n[2] = {n_tokens, q_heads};
    const Strides<2> by_q(n, strides), by_out(n, strides + 2);
    Span a, b;
    if (!span_of(q, 2, n, by_q.s, d, 2, &a) || !span_of(out, 2, n, by_out.s, d, 2, &b) ||
        !distinct(2, n, by_out.s, d) || !by_eight(q, 2, by_q.s, 2) || !aligned(out, 2) || a.meets(b))
        return LF_ERR_INVALID_ARG;
    const uint64_t need = workspace_of(sh, d, bits);
    if (need > 0 && !workspace) return LF_ERR_INVALID_ARG;
    if (workspace_bytes < need) return LF_ERR_SCRATCH_TOO_SMALL;
    if (n_tokens == 0) return LF_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    KvAttnParams p;
    std::memset(&p, 0, sizeof(p));
    int sms = 0;
    if ((st = device_info(s, &p.status, &sms)) != LF_OK || (st = kernel_limits()) != LF_OK) return st;
    p.q = q;
    p.out = out;
    p.q_row = by_q.s[0];
    p.q_head = by_q.s[1];
    p.o_wide = aligned(out, 8) && by_out.s[0] % 4 == 0 && by_out.s[1] % 4 == 0;
    p.o_row = by_out.s[0];
    p.o_head = by_out.s[1];
    p.k = static_cast<const uint8_t*>(k_cache);
    p.v = static_cast<const uint8_t*>(v_cache);
    p.k_par = static_cast<const uint8_t*>(k_par);
    p.v_par = static_cast<const uint8_t*>(v_par);
    p.table = table;
    p.plan = kv_plan_view(const_cast<void*>(plan), kv_plan_layout(n_seqs, n_tokens, n_global));
    p.part = static_cast<float*>(workspace);
    p.N = n_tokens;
    p.n_pages = n_pages;
    p.log_page = log2_of(page);
    p.max_pages = max_pages;
    p.kv_heads = kv_heads;
    p.group = q_heads / kv_heads;
    p.nsub = sh.nsub;
    p.gs = heads_of_unit(p.group, p.nsub);
    p.unit_rows = p.gs * sh.tpt;
    p.r = sh.r;
    p.n_global = n_global;
    p.G = sh.G;
    p.sl2 = static_cast<float>(double(scale) * kLog2e);
    p.sig = sh.sig_all;
    std::memcpy(p.dil, sh.dil, sizeof(p.dil));
    const bool half = dtype == LF_F16;
    int smem = 0;
    const bool pack = sh.tpt > 1;
    const AttnKernel kern = d == 64 ? (bits == 16 ? attn_kernel<64, 16>(half, p.unit_rows, pack, &smem)
                                                  : attn_kernel<64, 4>(half, p.unit_rows, pack, &smem))
                                    : (bits == 16 ? attn_kernel<128, 16>(half, p.unit_rows, pack, &smem)
                                                  : attn_kernel<128, 4>(half, p.unit_rows, pack, &smem));
    kern<<<p.G, kKvThreads, smem, s>>>(p);
    if (cudaGetLastError() != cudaSuccess) return LF_ERR_CUDA;
    if (!sh.cut) return LF_OK;
    const AttnKernel merge = d == 64 ? (half ? kv_merge_kernel<64, true> : kv_merge_kernel<64, false>)
                                     : (half ? kv_merge_kernel<128, true> : kv_merge_kernel<128, false>);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.G, p.unit_rows);
    cfg.blockDim = dim3(d);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, merge, p) == cudaSuccess ? LF_OK : LF_ERR_CUDA;
}

}  // extern "C"
