// kv_plan.cuh -- the plan of one step over the paged cache: which sequence
// and position each token row has, the sorted global tokens of each sequence,
// and how the attention's work is split over its CTAs.  Made on the device
// from device data (so a captured step replans itself on every replay) and
// read by all layers of the step with the same heads and window.
//
// The work sequence: tiles of token rows in order (a tile is one row, or, where
// a step has at least two rows a sequence, up to 16 / heads consecutive rows of
// a sequence, whose keys are nearly the same); per tile its units, one per kv
// head and group of at most 16 query heads of it; per unit first its
// own cost (kUnitKeys, in blocks), then its blocks of 64 or 128 keys, the
// window's before those of the sequence's global list.  CTA s of G' takes
// places [s W / G', (s + 1) W / G') of all W, so every CTA has the same work,
// give or take a block, however ragged the lengths are.  A unit that a range
// boundary cuts between its blocks leaves a partial state in every CTA that
// has a piece of it, and a merge kernel joins them.  G' = G unless a CTA would
// have fewer than kKvMinKeys keys: its start and a piece's end have a cost too.
//
// Units stay whole where cutting them would gain less than the merge costs
// (decided on the host from the window and the number of rows): a CTA takes
// the units that begin in its range, and nothing is merged.  (A global row,
// which sees every key, is then one CTA's work a head too: 16 single tokens at
// 32768, 12 heads of 64, window 256, take 8 us, and 308 where one of them is
// global.)
//
// Bound: latency (a few KB; 7 to 18 us for 1 to 64 sequences, 40 us for a
// prompt of 16384 rows, once for all layers of a step).  The global lists take
// one CTA per sequence; the rows, their prefix sum and the split one CTA in
// all, since each needs the whole of the one before, with what is searched
// held in shared memory.
#pragma once
#include "lf_common.cuh"
#include "ptx.cuh"

namespace lf {

constexpr int kKvMaxGlobal = 1024;     // global tokens per sequence (the lists are ranked in O(n^2))
constexpr int kKvMaxCtas = 640;
constexpr int kKvMinKeys = 256;        // keys (and units' costs) per CTA below which fewer CTAs take part
// Keys whose time a unit's beginning and end take.  Without it the CTAs that
// have the short rows at a prompt's start end last: 4096 rows that see all
// before them, 16 heads on 2 of 128, 863 us against 1514 (4 bits 766 : 1098; 512
// keys: 897 and 791); 4 sequences of up to 65536 over 4 bits 79.3 : 83.5.
constexpr int kUnitKeys = 256;
constexpr int kPlanThreads = 1024;
constexpr int kPlanSeqs = 4096, kPlanRows = 1024;  // up to which cu_tokens and the prefix sum are searched in shared memory
constexpr uint32_t kStatusBadCache = 4u;  // a row or page of a cache call outside its range (left out)
constexpr uint32_t kStatusBadPlan = 8u;   // a cache call with another plan than its arguments say

struct KvCut {
    int32_t row, unit;  // the unit that CTA s begins and a later one ends
    int32_t last;       // its last CTA; -1: CTA s begins no such unit
    int32_t tile;       // of its first row
};
struct KvStart {  // where a CTA's range starts, with the row's entries
    int32_t row, unit, blk, seq, pos, ng, lo, tile;
    int64_t n;  // what is left of the range from block blk on
};

struct KvPlan {  // views into the caller's plan buffer
    uint64_t* sig;       // [2]: of the rows (append), of rows and work (attention)
    int64_t* prefix;     // [N] places of the work sequence before each row
    KvStart* start;      // [G]
    KvCut* cut;          // [G]
    int32_t* row_seq;    // [N], -1: the row is none (behind the last sequence, or out of range)
    int32_t* row_pos;    // [N]
    int32_t* row_ng;     // [N] entries of the global list that may be its keys; -1: a global row alone (all keys)
    int32_t* row_tile;   // [N] rows of the tile that begins here, 0: none; from bit 8 which of them are global
    int32_t* row_lo;     // [N] tiles of several rows: the first position that a window of it reaches
    int32_t* g_count;    // [S]
    int32_t* g_list;     // [S][n_global] sorted, each once
};

struct KvShape {  // what a plan is made for
    int S, N, n_global, max_len;
    int q_heads, kv_heads, nsub, r, G;
    int tpt;             // most rows of a tile
    int block;           // keys per block
    int cut;             // 0: units stay whole
    int may_cut;         // 0: and would with any number of sequences
    int one_dil;         // all heads have dil[0]
    uint64_t sig_rows, sig_all;
    int32_t dil[kMaxHeads];
};

// Places in the plan buffer (bytes, 256-byte aligned).  What the attention
// reads before it has seen that the plan is its own lies at fixed places.
struct KvPlanLayout {
    size_t start, cut, prefix, seq, pos, ng, tile, lo, gcount, glist, total;
};
inline KvPlanLayout kv_plan_layout(int S, int N, int n_global) {
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    KvPlanLayout L;
    L.start = 256;
    L.cut = up(L.start + sizeof(KvStart) * kKvMaxCtas);
    L.prefix = up(L.cut + sizeof(KvCut) * kKvMaxCtas);
    L.seq = up(L.prefix + sizeof(int64_t) * size_t(N));
    L.pos = up(L.seq + sizeof(int32_t) * size_t(N));
    L.ng = up(L.pos + sizeof(int32_t) * size_t(N));
    L.tile = up(L.ng + sizeof(int32_t) * size_t(N));
    L.lo = up(L.tile + sizeof(int32_t) * size_t(N));
    L.gcount = up(L.lo + sizeof(int32_t) * size_t(N));
    L.glist = up(L.gcount + sizeof(int32_t) * size_t(S));
    L.total = up(L.glist + sizeof(int32_t) * size_t(S) * n_global);
    return L;
}
inline KvPlan kv_plan_view(void* buf, const KvPlanLayout& L) {
    uint8_t* b = static_cast<uint8_t*>(buf);
    KvPlan p;
    p.sig = reinterpret_cast<uint64_t*>(b);
    p.prefix = reinterpret_cast<int64_t*>(b + L.prefix);
    p.start = reinterpret_cast<KvStart*>(b + L.start);
    p.cut = reinterpret_cast<KvCut*>(b + L.cut);
    p.row_seq = reinterpret_cast<int32_t*>(b + L.seq);
    p.row_pos = reinterpret_cast<int32_t*>(b + L.pos);
    p.row_ng = reinterpret_cast<int32_t*>(b + L.ng);
    p.row_tile = reinterpret_cast<int32_t*>(b + L.tile);
    p.row_lo = reinterpret_cast<int32_t*>(b + L.lo);
    p.g_count = reinterpret_cast<int32_t*>(b + L.gcount);
    p.g_list = reinterpret_cast<int32_t*>(b + L.glist);
    return p;
}

// A unit's keys: window key n < n_win sits at position first + n * step, key
// n_win + a is entry a of the global list (an entry inside the window is left
// out there, so each key counts once).
struct KvKeys {
    int first, step, n_win, n;
    __host__ __device__ KvKeys(int pos, int ng_row, int r, int dil) {
        step = ng_row < 0 ? 1 : dil;
        const int back = ng_row < 0 ? pos : (pos / dil < r ? pos / dil : r);
        n_win = back + 1;
        first = pos - back * step;
        n = n_win + (ng_row < 0 ? 0 : ng_row);
    }
    // A tile's: positions lo .. last, then the first ng entries of the list.
    __host__ __device__ KvKeys(int lo, int last, int ng) : first(lo), step(1), n_win(last - lo + 1), n(n_win + ng) {}
    __host__ __device__ int blocks(int block) const { return (n + block - 1) / block; }
};

// Sorts a sequence's global tokens, each once.  grid: S; smem: 2 n_global ints.
__global__ void __launch_bounds__(256) kv_plan_globals_kernel(const int32_t* gidx, int n_global, int max_len, KvPlan p,
                                                              uint32_t* status) {
    extern __shared__ int32_t s_g[];
    int32_t* s_keep = s_g + n_global;
    const int s = blockIdx.x;
    for (int i = threadIdx.x; i < n_global; i += 256) {
        const int g = gidx[int64_t(s) * n_global + i];
        s_g[i] = g;
        if (g < 0 || g >= max_len) atomicOr(status, kStatusBadGlobal);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n_global; i += 256) {
        const int g = s_g[i];
        bool keep = g >= 0 && g < max_len;
        for (int j = 0; j < i && keep; ++j) keep = s_g[j] != g;
        s_keep[i] = keep;
    }
    __syncthreads();
    int kept = 0;
    for (int i = threadIdx.x; i < n_global; i += 256) {
        if (!s_keep[i]) continue;
        ++kept;
        int rank = 0;
        for (int j = 0; j < n_global; ++j) rank += s_keep[j] && s_g[j] < s_g[i];
        p.g_list[int64_t(s) * n_global + rank] = s_g[i];
    }
    // the last entry's rank + 1 is the count
    __shared__ int s_n;
    if (threadIdx.x == 0) s_n = 0;
    __syncthreads();
    if (kept) atomicAdd(&s_n, kept);
    __syncthreads();
    if (threadIdx.x == 0) p.g_count[s] = s_n;
}

// Rows, prefix sum and split.  One CTA.
__global__ void __launch_bounds__(kPlanThreads) kv_plan_rows_kernel(const int32_t* cu, const int32_t* context,
                                                                    const __grid_constant__ KvShape sh, KvPlan p,
                                                                    uint32_t* status) {
    __shared__ int32_t s_cu[kPlanSeqs + 1];
    __shared__ int64_t s_prefix[kPlanRows], s_bound[kKvMaxCtas + 1], s_warp[32], s_carry;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) s_carry = 0;
    bool falls = false;
    for (int s = tid; s <= sh.S; s += kPlanThreads) {
        const int c = cu[s];
        if (s <= kPlanSeqs) s_cu[s] = c;
        falls |= s > 0 && c < cu[s - 1];
        if (s == 0 ? c != 0 : c < cu[s - 1]) atomicOr(status, kStatusBadCache);
        if (s == sh.S && c > sh.N) atomicOr(status, kStatusBadCache);
    }
    const bool none = __syncthreads_or(falls);  // else two sequences, and two tiles, could have one row
    const int32_t* cus = sh.S <= kPlanSeqs ? s_cu : cu;
    const int64_t* prefix = sh.N <= kPlanRows ? s_prefix : p.prefix;
    const int unit_cost = kUnitKeys / sh.block;
    auto blocks_of = [&](int pos, int ng, int lo, int tile, int h) {
        return unit_cost + (sh.tpt > 1 ? KvKeys(lo, pos + (tile & 255) - 1, ng) : KvKeys(pos, ng, sh.r, sh.dil[h])).blocks(sh.block);
    };
    for (int n0 = 0; n0 < sh.N; n0 += kPlanThreads) {
        const int n = n0 + tid;
        int64_t blocks = 0;
        if (n < sh.N) {
            int lo = 0, hi = sh.S;  // the last s with cu[s] <= n
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cus[mid] <= n) lo = mid;
                else hi = mid;
            }
            const int c0 = cus[lo], c1 = cus[lo + 1];
            int seq = -1, pos = 0, ng = 0;
            if (!none && c0 >= 0 && c0 <= n && n < c1) {
                const int before = context[lo];
                const int64_t at = int64_t(before) + (n - c0);
                if (before >= 0 && at < sh.max_len) {
                    seq = lo;
                    pos = static_cast<int>(at);
                } else {
                    atomicOr(status, kStatusBadCache);
                }
            }
            int tile = 0, first = 0;
            if (seq >= 0 && (n - c0) % sh.tpt == 0) {
                const int m = min(min(sh.tpt, min(c1, sh.N) - n), sh.max_len - pos);  // rows past the table are none
                const int32_t* g = p.g_list + int64_t(seq) * sh.n_global;
                const int cnt = sh.n_global > 0 ? p.g_count[seq] : 0;
                auto below = [&](int x) {  // entries of the list below x
                    int a = 0, b = cnt;
                    while (a < b) {
                        const int mid = (a + b) >> 1;
                        if (g[mid] < x) a = mid + 1;
                        else b = mid;
                    }
                    return a;
                };
                tile = m;
                if (sh.tpt == 1) {
                    ng = below(pos);
                    if (ng < cnt && g[ng] == pos) ng = -1;
                } else {  // the rows' windows together, and the entries behind the last of them
                    for (int a = cnt > 0 ? below(pos) : 0; a < cnt && g[a] < pos + m; ++a) tile |= 256 << (g[a] - pos);
                    const uint32_t others = ~(tile >> 8) & ((1u << m) - 1);  // rows that are not global
                    first = others + 1 == 1u << m ? max(0, pos - sh.r) : 0;
                    const int top = others ? max(0, pos + 31 - __clz(others) - sh.r) : 0;
                    ng = cnt > 0 && top > 0 ? below(top) : 0;
                }
                if (sh.one_dil) blocks = int64_t(sh.kv_heads) * blocks_of(pos, ng, first, tile, 0);
                else
                    for (int h = 0; h < sh.kv_heads; ++h) blocks += blocks_of(pos, ng, first, tile, h);
                blocks *= sh.nsub;
            }
            p.row_tile[n] = tile;
            p.row_lo[n] = first;
            p.row_seq[n] = seq;
            p.row_pos[n] = pos;
            p.row_ng[n] = ng;
        }
        int64_t sum = blocks;  // inclusive scan over the CTA
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t t = __shfl_up_sync(~0u, sum, o);
            if (lane >= o) sum += t;
        }
        if (lane == 31) s_warp[warp] = sum;
        __syncthreads();
        if (warp == 0) {
            int64_t w = s_warp[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t t = __shfl_up_sync(~0u, w, o);
                if (lane >= o) w += t;
            }
            s_warp[lane] = w;
        }
        __syncthreads();
        const int64_t before = s_carry + (warp ? s_warp[warp - 1] : 0) + sum - blocks;
        if (n < sh.N) {
            p.prefix[n] = before;
            if (n < kPlanRows) s_prefix[n] = before;
        }
        __syncthreads();
        if (tid == kPlanThreads - 1) s_carry = before + blocks;
        __syncthreads();
    }
    const int64_t W = s_carry;  // in blocks, the units' costs with them
    if (tid == 0) {
        p.sig[0] = sh.sig_rows;
        p.sig[1] = sh.sig_all;
    }
    // The split.  Place x of the sequence: its row, unit, and block of the unit.
    const int64_t wide = sh.cut ? (W * sh.block + kKvMinKeys - 1) / kKvMinKeys : W;
    const int64_t G = wide < sh.G ? wide : sh.G;  // no CTA below G has an empty range
    auto locate = [&](int64_t x, KvStart& at, int64_t& unit_first, int64_t& unit_end) {
        int lo = 0, hi = sh.N;  // the last row with prefix <= x (rows without blocks are passed over)
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (prefix[mid] <= x) lo = mid;
            else hi = mid;
        }
        int64_t left = x - prefix[lo];
        at.row = lo;
        at.seq = p.row_seq[lo];
        at.pos = p.row_pos[lo];
        at.ng = p.row_ng[lo];
        at.lo = p.row_lo[lo];
        at.tile = p.row_tile[lo];
        int unit = 0, nb = 1;
        for (int h = 0; h < sh.kv_heads; ++h) {
            nb = blocks_of(at.pos, at.ng, at.lo, at.tile, h);
            const int64_t all = int64_t(nb) * sh.nsub * (sh.one_dil ? sh.kv_heads : 1);
            if (left < all) {
                unit = h * sh.nsub + static_cast<int>(left / nb);
                left %= nb;
                break;
            }
            left -= all;
        }
        at.unit = unit;
        at.blk = static_cast<int>(left > unit_cost ? left - unit_cost : 0);
        at.n = left < unit_cost ? left - unit_cost : 0;  // of the unit's own cost, what is still to come
        unit_first = x - left;
        unit_end = unit_first + nb;
    };
    for (int s = tid; s <= G; s += kPlanThreads) {  // where the CTAs' ranges start
        int64_t x = G > 0 ? s * W / G : 0;
        if (!sh.cut && x < W) {  // the first unit boundary at or behind x
            KvStart at;
            int64_t first, end;
            locate(x, at, first, end);
            if (first < x) x = end;
        }
        s_bound[s] = x;
    }
    __syncthreads();
    for (int s = tid; s < sh.G; s += kPlanThreads) {
        KvStart at{0, 0, 0, 0, 0, 0, 0, 0, 0};
        KvCut cut{0, 0, -1, 0};
        if (s < G && s_bound[s] < s_bound[s + 1]) {
            const int64_t x0 = s_bound[s], x1 = s_bound[s + 1];
            int64_t first, end;
            locate(x0, at, first, end);
            at.n += x1 - x0;
            if (sh.cut) {
                KvStart last;
                locate(x1 - 1, last, first, end);
                if (first + unit_cost >= x0 && first + unit_cost < x1 && end > x1) {
                    cut.row = last.row;
                    cut.unit = last.unit;
                    cut.tile = last.tile;
                    cut.last = static_cast<int>((end * G - 1) / W);  // the CTA that has block end - 1
                }
            }
        }
        p.start[s] = at;
        p.cut[s] = cut;
    }
}

}  // namespace lf
