// A paged cache: new tokens' keys and values on their way into it, with the
// rotation of positions, and attention of those tokens over it.
//
// A sequence holds ctx tokens that every new one sees, and behind them the new
// ones; new token i sees those that its bits name (a tree of drafts), or without
// bits those up to itself. Query heads of a group stand side by side as rows, so
// that a tile of keys is read once for all of them, and the keys of a sequence
// are cut into parts for as many workgroups as the chip holds, whose results
// (maximum, sum and o from nothing) are joined by a second kernel.
#include <algorithm>
#include <type_traits>

#include "kda_attn.h"
#include "kda_launch.h"

namespace kda {

namespace {

size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

// Where token `row` of a sequence lies in the cache: its row over all pages, or
// -1 where the table names no page for it.
struct Pages {
    const int32_t* table;   // [N, width]
    int width, page, shift, count;   // shift: page = 1 << shift, or -1
    __device__ __forceinline__ int row(int seq, int row) const {
        const int i = shift >= 0 ? row >> shift : row / page;
        if (row < 0 || i >= width) return -1;
        const int at = table[(size_t)seq * width + i];
        return (unsigned)at < (unsigned)count ? at * page + (row - i * page) : -1;
    }
};

Pages make_pages(const PagedArgs& a) {
    int shift = -1;
    if ((a.page_size & (a.page_size - 1)) == 0) shift = __builtin_ctz(a.page_size);
    return Pages{a.table, a.width, a.page_size, shift, a.num_pages};
}

// ---------------------------------------------------------------- append

struct AppendParams {
    const void *q, *k, *v;
    void *q_out, *Kp, *Vp;
    const int32_t *pos, *ctx;
    const float* freqs;
    Pages pages;
    SeqMap map;
    int rows, Hq, Hkv, rot;   // rows: tokens over the batch
};

// sequence of a token, and its place there; false behind the last sequence
__device__ __forceinline__ bool token_place(const SeqMap& m, int t, int& seq, int& i) {
    if (m.cu == nullptr) {
        seq = t / m.T;
        i = t % m.T;
        return true;
    }
    int lo = 0, hi = m.N;   // the number of offsets at or before t, less one
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (seq_offset(m, mid + 1) <= t) lo = mid + 1; else hi = mid;
    }
    seq = lo;
    if (lo >= m.N) return false;
    i = t - seq_offset(m, lo);
    return i >= 0;
}

// A wave takes a token: cosines and sines of its angles once, then the rows of
// all its heads, two pieces of 16 bytes a lane that hold each other's partners.
// Angles are formed and reduced to one turn in 64 bits (position and frequency
// are exact, their product is at positions where 32 bits have no fraction left).
template <class T, int D> __global__ void __launch_bounds__(256) paged_append_kernel(AppendParams p, bool neighbours) {
    lds_poison(0);
    __shared__ float s_cos[4][64], s_sin[4][64];
    constexpr int V = 16 / (int)sizeof(T), U = D / (2 * V);   // elements of a piece, units of two of them in a row
    const int w = threadIdx.x / WAVE, lane = threadIdx.x % WAVE;
    const int t = blockIdx.x * 4 + w;
    if (t >= p.rows) return;
    int seq, i;
    if (!token_place(p.map, t, seq, i)) return;
    const int ctx = p.ctx[seq];
    const long row = (long)ctx + i;
    const int slot = ctx < 0 || row > 0x7fffffffL ? -1 : p.pages.row(seq, (int)row);
    const int half = p.rot / 2;
    if (lane < half) {
        const double turns = (double)(p.pos ? p.pos[t] : row) * (double)p.freqs[lane] * 0.15915494309189535;
        float sn, cs;
        sincospif(2.f * (float)(turns - rint(turns)), &sn, &cs);
        s_cos[w][lane] = cs;
        s_sin[w][lane] = sn;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int rot_units = half / V;
    const int hq = p.q ? p.Hq : 0, heads = hq + 2 * p.Hkv;
    for (int e = lane; e < heads * U; e += WAVE) {
        const int h = e / U, u = e % U;
        const T* from;
        T* to = nullptr;
        bool turn = true;
        if (h < hq) {
            const size_t at = ((size_t)t * p.Hq + h) * D;
            from = static_cast<const T*>(p.q) + at;
            to = static_cast<T*>(p.q_out) + at;
        } else {
            const bool isv = h >= hq + p.Hkv;
            const int hk = h - hq - (isv ? p.Hkv : 0);
            from = static_cast<const T*>(isv ? p.v : p.k) + ((size_t)t * p.Hkv + hk) * D;
            if (slot < 0) continue;
            to = static_cast<T*>(isv ? p.Vp : p.Kp) + ((size_t)slot * p.Hkv + hk) * D;
            turn = !isv;
        }
        if (ctx < 0) {   // left out: only q's rows are written
            const uint4 z = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(to + 2 * u * V) = z;
            *reinterpret_cast<uint4*>(to + (2 * u + 1) * V) = z;
            continue;
        }
        turn = turn && u < rot_units;
        const bool halves = !neighbours && u < rot_units;
        const int a = (halves ? u : 2 * u) * V, b = halves ? a + half : a + V;
        uint4 x = *reinterpret_cast<const uint4*>(from + a), y = *reinterpret_cast<const uint4*>(from + b);
        if (turn) {
            T xs[V], ys[V];
            __builtin_memcpy(xs, &x, 16);
            __builtin_memcpy(ys, &y, 16);
            if (halves) {
#pragma unroll
                for (int m = 0; m < V; ++m) {
                    const float c = s_cos[w][a + m], s = s_sin[w][a + m], f = from_el(xs[m]), g = from_el(ys[m]);
                    store1(xs + m, f * c - g * s);
                    store1(ys + m, f * s + g * c);
                }
            } else {
#pragma unroll
                for (int m = 0; m < V; m += 2) {
                    const float c = s_cos[w][(a + m) / 2], s = s_sin[w][(a + m) / 2], f = from_el(xs[m]), g = from_el(xs[m + 1]);
                    store1(xs + m, f * c - g * s);
                    store1(xs + m + 1, f * s + g * c);
                    const float c2 = s_cos[w][(b + m) / 2], s2 = s_sin[w][(b + m) / 2], f2 = from_el(ys[m]), g2 = from_el(ys[m + 1]);
                    store1(ys + m, f2 * c2 - g2 * s2);
                    store1(ys + m + 1, f2 * s2 + g2 * c2);
                }
            }
            __builtin_memcpy(&x, xs, 16);
            __builtin_memcpy(&y, ys, 16);
        }
        *reinterpret_cast<uint4*>(to + a) = x;
        *reinterpret_cast<uint4*>(to + b) = y;
    }
}

// ---------------------------------------------------------------- attention

struct AttnParams {
    const void *q, *Kp, *Vp;
    const int32_t *ctx, *tree;
    void* out;
    float* lse;
    Pages pages;
    SeqMap map;
    int Hq, Hkv, G, words;
    long capacity;          // of a sequence's pages
    float scale;
    int blocks;             // blocks of rows over all sequences
    int wgs;                // workgroups that share the keys, or 0: one for each item
    int2* span;             // [item]: the first and last workgroup of an item that is shared
    float *po, *pml;        // parts: [2 * wgs][R][D], [2 * wgs][R][2]
};

constexpr int MAX_BLOCKS = 1024;   // of a call whose keys are shared out
constexpr int WGS = 512;           // two for each CU, what LDS takes

// A block of R rows (token, head of a group) of one sequence.
struct RowBlock {
    int seq, r0, rows, n;   // sequence, first row, rows of the sequence, its tokens
    long t0;                // its first token, flattened over the batch
};
__host__ __device__ inline long row_blocks_bound(int T, int N, int G, int R, bool packed) {
    return packed ? (long)T * G / R + N + 1 : (long)N * (((long)T * G + R - 1) / R);
}
__device__ __forceinline__ bool row_block(const SeqMap& m, int G, int R, int v, RowBlock& b) {
    if (m.cu == nullptr) {
        const int nb = (m.T * G + R - 1) / R;
        b.seq = v / nb;
        b.r0 = v % nb * R;
        b.n = m.T;
        b.t0 = (long)b.seq * m.T;
    } else {
        int lo = 0, hi = m.N - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (seq_offset(m, mid) * G / R + mid <= v) lo = mid; else hi = mid - 1;
        }
        const int c0 = seq_offset(m, lo);
        b.seq = lo;
        b.r0 = (v - c0 * G / R - lo) * R;
        b.n = max(seq_offset(m, lo + 1) - c0, 0);
        b.t0 = c0;
    }
    b.rows = b.n * G;
    return b.r0 >= 0 && b.r0 < b.rows;
}
// keys that a block's rows may see
__device__ __forceinline__ int keys_of(const AttnParams& p, const RowBlock& b, int R) {
    const int ctx = p.ctx[b.seq];
    if (ctx < 0) return 0;
    return (int)min((long)ctx + (p.tree ? b.n : min(b.n, (b.r0 + R - 1) / p.G + 1)), p.capacity);
}

// Rows' tiles of 32 a workgroup has (RW), and the groups of waves (KS = 4 / RW) that
// take every KS-th tile of keys each.
template <class T, int RW> struct Shape {
    static constexpr int KS = 4 / RW, R = 32 * RW, KT = sizeof(T) == 2 && RW == 4 ? 64 : 32, KB = KS * KT;
    static constexpr int NB = RW == 1 ? 1 : 2;   // buffers: a wave by itself needs no second one
};
template <class T, int D, int RW> constexpr size_t attn_lds() {
    using S = Shape<T, RW>;
    const size_t tiles = sizeof(T) * S::KS * S::NB * 2 * S::KT * tile_stride<T>(D);
    const size_t join = S::KS > 1 ? sizeof(float) * 4 * 64 * (16 * (D / 32) + 2) : 0;
    return tiles > join ? tiles : join;
}

template <class T, int D, int RW> __global__ void __launch_bounds__(256) paged_attn_kernel(AttnParams p) {
    using S = Shape<T, RW>;
    constexpr int KS = S::KS, R = S::R, KT = S::KT, KB = S::KB, NB = S::NB, NX = KT / 32, GT = 64 * RW;
    constexpr int ST = tile_stride<T>(D), KD = D / 16, MD = D / 32, PER = 16 / (int)sizeof(T), CPR = D / PER, NL = KT * CPR / GT;
    using V8 = typename Frag<T>::V;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ int s_units[MAX_BLOCKS], s_first[MAX_BLOCKS + 1];
    lds_poison((uint32_t)attn_lds<T, D, RW>());
    const int tid = threadIdx.x, lane = tid % WAVE, w = wave_id(), n = lane & 31, h2 = lane >> 5;
    const int wr = w % RW, wk = w / RW, gt = tid - wk * GT;
    T* const tiles = reinterpret_cast<T*>(smem) + (size_t)wk * NB * 2 * KT * ST;   // [buffer][k, v][KT][ST]
    const float c = fabsf(p.scale) * LOG2E;
    const size_t rs = (size_t)p.Hkv * D;

    // this workgroup's units (KB keys of one item): [u, end)
    int v = 0, hk = 0, it0 = 0;
    long u = 0, end = 0, per = 0;
    if (p.wgs) {
        int sum = 0;   // of this thread's blocks: MAX_BLOCKS / 256 neighbours
        constexpr int B = MAX_BLOCKS / 256;
        int mine[B];
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const int b = tid * B + i;
            RowBlock rb;
            mine[i] = 0;
            if (b < p.blocks && row_block(p.map, p.G, R, b, rb)) mine[i] = max((keys_of(p, rb, R) + KB - 1) / KB, 1);
            sum += mine[i];
        }
        int before = sum;
#pragma unroll
        for (int o = 1; o < WAVE; o *= 2) {
            const int y = __shfl_up(before, o, WAVE);
            if (lane >= o) before += y;
        }
        __shared__ int s_wave[4];
        if (lane == 63) s_wave[w] = before;
        __syncthreads();
        before -= sum;
        for (int i = 0; i < w; ++i) before += s_wave[i];
#pragma unroll
        for (int i = 0; i < B; ++i) {
            s_units[tid * B + i] = mine[i];
            s_first[tid * B + i] = before;
            before += mine[i];
        }
        if (tid == 255) s_first[MAX_BLOCKS] = before;
        __syncthreads();
        const long total = (long)s_first[MAX_BLOCKS] * p.Hkv;
        per = (total + p.wgs - 1) / p.wgs;
        u = per * blockIdx.x;
        end = min(u + per, total);
        if (u >= end) return;
        int lo = 0, hi = p.blocks - 1;   // the block that holds unit u
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((long)s_first[mid] * p.Hkv <= u) lo = mid; else hi = mid - 1;
        }
        // (of blocks with the same first unit the search ends at the last, the one that is not empty)
        v = __builtin_amdgcn_readfirstlane(lo);
        const int rem = (int)(u - (long)s_first[v] * p.Hkv), un = s_units[v];
        hk = __builtin_amdgcn_readfirstlane(rem / un);
        it0 = __builtin_amdgcn_readfirstlane(rem % un);
    } else {
        v = blockIdx.x / p.Hkv;
        hk = blockIdx.x % p.Hkv;
        u = 0;
        end = 1;
    }

    for (; u < end && v < p.blocks; it0 = 0) {
        RowBlock b;
        if (!row_block(p.map, p.G, R, v, b)) {   // an empty number of a packed batch
            if (!p.wgs) return;
            ++v;
            continue;
        }
        const int ctx = p.ctx[b.seq], keys = keys_of(p, b, R);
        const int units = max((keys + KB - 1) / KB, 1);
        const int it1 = p.wgs ? (int)min((long)units, it0 + (end - u)) : units;
        const bool whole = it0 == 0 && it1 == units;
        const int rr = b.r0 + 32 * wr + n;
        const bool live = rr < b.rows;
        const int tok = (live ? rr : 0) / p.G, head = hk * p.G + (live ? rr : 0) % p.G;
        const size_t q_at = ((size_t)(b.t0 + tok) * p.Hq + head) * D;

        V8 qf[KD];
#pragma unroll
        for (int ks = 0; ks < KD; ++ks) {
            qf[ks] = load8<T>(static_cast<const T*>(p.q) + q_at + 8 * h2 + 16 * ks, live);
            if (p.scale < 0.f) qf[ks] = -qf[ks];   // exact, so that maxima scale as they stand
        }
        const T* const K = static_cast<const T*>(p.Kp) + (size_t)hk * D;
        const T* const V = static_cast<const T*>(p.Vp) + (size_t)hk * D;
        const int32_t* const bits = p.tree ? p.tree + (size_t)(b.t0 + tok) * p.words : nullptr;

        // the row in the cache of key (tile's first + lane), or -1
        auto lookup = [&](int it) {
            const int j = (it * KS + wk) * KT + lane;
            return lane < KT && j < keys ? p.pages.row(b.seq, j) : -1;
        };
        u32x4 rk[NL], rv[NL];
        auto fetch = [&](int where) {
#pragma unroll
            for (int m = 0; m < NL; ++m) {
                const int e = gt + m * GT, at = max(__shfl(where, e / CPR, WAVE), 0);
                const size_t o = (size_t)at * rs + e % CPR * PER;
                rk[m] = *reinterpret_cast<const u32x4*>(K + o);
                rv[m] = *reinterpret_cast<const u32x4*>(V + o);
            }
        };
        auto put = [&](T* t, uint64_t held, bool full) {
#pragma unroll
            for (int m = 0; m < NL; ++m) {
                const int e = gt + m * GT, row = e / CPR, at = row * ST + e % CPR * PER;
                if (!full && !(held >> row & 1)) {   // what lies there is not this sequence's
                    rk[m] = u32x4{0u, 0u, 0u, 0u};
                    rv[m] = u32x4{0u, 0u, 0u, 0u};
                }
                *reinterpret_cast<u32x4*>(t + at) = rk[m];
                *reinterpret_cast<u32x4*>(t + KT * ST + at) = rv[m];
            }
        };
        // which of the 32 keys from j0 on this lane's row sees
        auto visible = [&](int j0) -> uint32_t {
            const int d = j0 - ctx;   // among the new tokens
            if (bits == nullptr) {
                const int m = min(max(tok - d + 1, 0), 32);
                return m == 32 ? ~0u : (1u << m) - 1u;
            }
            if (d <= -32) return ~0u;
            if (d < 0) return ((1u << -d) - 1u) | (uint32_t)bits[0] << -d;
            const int at = d >> 5, sh = d & 31;
            const uint32_t x = at < p.words ? (uint32_t)bits[at] : 0u;
            const uint32_t y = sh && at + 1 < p.words ? (uint32_t)bits[at + 1] << (32 - sh) : 0u;
            return x >> sh | y;
        };

        f32x16 O[MD];
#pragma unroll
        for (int m = 0; m < MD; ++m) O[m] = zero16();
        float top = -INFINITY, sum = 0.f;   // sum: this lane's half of the keys

        auto tile = [&](const T* tk, const T* tv, int j0, uint64_t held, auto masked) {
            f32x16 s[NX];
#pragma unroll
            for (int x = 0; x < NX; ++x) {
                s[x] = zero16();
#pragma unroll
                for (int ks = 0; ks < KD; ++ks) s[x] = mma32(nat32<T>(tk, ST, 32 * x, 16 * ks, n, h2), qf[ks], s[x]);
            }
            if constexpr (masked.value) {
#pragma unroll
                for (int x = 0; x < NX; ++x) {
                    const uint32_t see = (visible(j0 + 32 * x) & (uint32_t)(held >> 32 * x)) >> 4 * h2;
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[x][r] = see >> result_row(r, 0) & 1u ? s[x][r] * c : -INFINITY;
                }
            }
            const float f = masked.value ? 1.f : c;   // what is left to scale
            float mt = tree_max(s[0]);
#pragma unroll
            for (int x = 1; x < NX; ++x) mt = __builtin_elementwise_maximum(mt, tree_max(s[x]));
            mt = swap_max(mt * f);
            // the subtracted maximum may lag behind by 2^8: most tiles leave o as it is
            if (__any(mt > top + 8.f || (top == -INFINITY && mt > top))) {
                const float next = fmaxf(top, mt);
                const float down = next == -INFINITY ? 1.f : fast_exp2(top - next);
                top = next;
                sum *= down;
#pragma unroll
                for (int m = 0; m < MD; ++m)
#pragma unroll
                    for (int r = 0; r < 16; ++r) O[m][r] *= down;
            }
            const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
            for (int x = 0; x < NX; ++x) {
                float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    s[x][r] = fast_exp2(fmaf(s[x][r], f, -base));
                    part[r & 3] += s[x][r];
                }
                sum += (part[0] + part[1]) + (part[2] + part[3]);
            }
#pragma unroll
            for (int kb = 0; kb < KT / 16; ++kb) {
                const V8 pf = rows16<T>(s[kb / 2], kb % 2);
#pragma unroll
                for (int m = 0; m < MD; ++m) O[m] = mma32(tr32(tv, ST, 16 * kb, 32 * m, lane), pf, O[m]);
            }
        };

        int where = lookup(it0);
        uint64_t held = __ballot(where >= 0);
        constexpr uint64_t ALL = KT == 64 ? ~0ull : 0xffffffffull;
        __syncthreads();   // the last item's tiles and joins are done with
        fetch(where);
        int where_next = it0 + 1 < it1 ? lookup(it0 + 1) : -1;
        for (int it = it0; it < it1; ++it) {
            T* const t = tiles + (size_t)(NB == 2 ? (it & 1) : 0) * 2 * KT * ST;
            put(t, held, held == ALL);
            if constexpr (RW == 1) {   // the tile is this wave's own: its reads and writes are in order
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
            } else {
                __syncthreads();
            }
            const uint64_t now = held;
            if (it + 1 < it1) {
                held = __ballot(where_next >= 0);
                fetch(where_next);
                where_next = it + 2 < it1 ? lookup(it + 2) : -1;
            }
            const int j0 = (it * KS + wk) * KT;
            if (now) {
                const int last_seen = bits ? ctx - 1 : ctx + (b.r0 + 32 * wr) / p.G;   // by every row of this wave
                if (now == ALL && j0 + KT - 1 <= last_seen) tile(t, t + KT * ST, j0, now, std::false_type());
                else tile(t, t + KT * ST, j0, now, std::true_type());
            }
            if constexpr (RW == 1) {
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
            }
        }
        sum = swap_sum(sum);
        // An Inf or NaN in v at a key that a tile holds but a row does not see has entered
        // that row as 0 * v. Rows that are not finite are formed again, one key at a time,
        // from the keys that they see.
        float probe = 0.f;
#pragma unroll
        for (int m = 0; m < MD; ++m)
#pragma unroll
            for (int r = 0; r < 16; ++r) probe += O[m][r] * 0.f;
        if (__any(live && probe != 0.f)) {
            const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
            for (int m = 0; m < MD; ++m) O[m] = zero16();
            for (int it = it0; it < it1; ++it) {
                const int rows = lookup(it), j0 = (it * KS + wk) * KT;
                for (int j = 0; j < KT; ++j) {
                    const int at = __shfl(rows, j, WAVE);
                    const bool in = live && at >= 0 && (visible(j0 + (j & 32)) >> (j & 31) & 1u);
                    if (!__any(in)) continue;
                    const T* const kr = K + (size_t)max(at, 0) * rs;
                    const T* const vr = V + (size_t)max(at, 0) * rs;
                    float dot = 0.f;
                    for (int x = 0; x < D; x += 8) {
                        const f32x8 y = widen(load8<T>(static_cast<const T*>(p.q) + q_at + x, true)) * widen(load8<T>(kr + x, true));
                        dot += ((y[0] + y[1]) + (y[2] + y[3])) + ((y[4] + y[5]) + (y[6] + y[7]));
                    }
                    const float e = fast_exp2(dot * (p.scale * LOG2E) - base);
                    if (!in) continue;
#pragma unroll
                    for (int m = 0; m < MD; ++m)
#pragma unroll
                        for (int r = 0; r < 16; ++r) O[m][r] += e * from_el(vr[32 * m + result_row(r, h2)]);
                }
            }
        }
        if constexpr (KS > 1) {   // the groups' shares, in the tiles' place: [wave][value][lane]
            float* const join = reinterpret_cast<float*>(smem) + (size_t)w * (16 * MD + 2) * 64 + lane;
            __syncthreads();
            if (wk) {
                join[0] = top;
                join[64] = sum;
#pragma unroll
                for (int m = 0; m < MD; ++m)
#pragma unroll
                    for (int r = 0; r < 16; ++r) join[(2 + 16 * m + r) * 64] = O[m][r];
            }
            __syncthreads();
            if (wk == 0) {
#pragma unroll
                for (int y = 1; y < KS; ++y) {
                    const float* other = join + (size_t)y * RW * (16 * MD + 2) * 64;
                    const float next = fmaxf(top, other[0]), base = next == -INFINITY ? 0.f : next;
                    const float fa = fast_exp2(top - base), fb = fast_exp2(other[0] - base);
                    top = next;
                    sum = sum * fa + other[64] * fb;
#pragma unroll
                    for (int m = 0; m < MD; ++m)
#pragma unroll
                        for (int r = 0; r < 16; ++r) O[m][r] = O[m][r] * fa + other[(2 + 16 * m + r) * 64] * fb;
                }
            }
        }
        if (wk == 0 && live) {
            if (whole) {
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                T* out = static_cast<T*>(p.out) + q_at;
#pragma unroll
                for (int m = 0; m < MD; ++m) store_tile<T>(out + 32 * m, O[m], inv, h2);
                if (p.lse && h2 == 0) p.lse[(size_t)(b.t0 + tok) * p.Hq + head] = (top + log2f(sum)) * LN2;
            } else {
                const size_t slot = ((size_t)2 * blockIdx.x + (it0 == 0 ? 1 : 0)) * R + 32 * wr + n;
                float* po = p.po + slot * D + 4 * h2;
#pragma unroll
                for (int m = 0; m < MD; ++m)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        *reinterpret_cast<f32x4*>(po + 32 * m + 8 * r) = f32x4{O[m][4 * r], O[m][4 * r + 1], O[m][4 * r + 2], O[m][4 * r + 3]};
                if (h2 == 0) {
                    p.pml[2 * slot] = top;
                    p.pml[2 * slot + 1] = sum;
                }
            }
        }
        if (p.wgs && it0 == 0 && tid == 0)
            p.span[v * p.Hkv + hk] = make_int2((int)blockIdx.x, (int)((u + units - 1) / per));
        u += it1 - it0;
        if (++hk == p.Hkv || !p.wgs) {
            hk = 0;
            ++v;
        }
    }
}

// Joins the parts of one row: four values a thread, the parts spread over the rest of
// the workgroup.
template <class T, int D, int RW> __global__ void __launch_bounds__(256) paged_join_kernel(AttnParams p) {
    lds_poison(0);
    constexpr int R = Shape<T, RW>::R, CG = D / 4, RG = 256 / CG;
    __shared__ float s_l[RG];
    __shared__ __align__(16) float s_o[RG][D];
    const int item = blockIdx.x / R, row = blockIdx.x % R, v = item / p.Hkv, hk = item % p.Hkv;
    RowBlock b;
    if (!row_block(p.map, p.G, R, v, b) || b.r0 + row >= b.rows) return;
    const int2 span = p.span[item];
    if (span.x == span.y) return;
    const int parts = span.y - span.x + 1;
    auto slot = [&](int y) { return ((size_t)2 * (span.x + y) + (y == 0 ? 1 : 0)) * R + row; };
    const int cg = threadIdx.x % CG, rg = threadIdx.x / CG;
    float m = -INFINITY;
    for (int y = 0; y < parts; ++y) m = fmaxf(m, p.pml[2 * slot(y)]);
    const float base = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    f32x4 acc = zero4();
    for (int y = rg; y < parts; y += RG) {
        const float f = fast_exp2(p.pml[2 * slot(y)] - base);
        l += f * p.pml[2 * slot(y) + 1];
        acc += *reinterpret_cast<const f32x4*>(p.po + slot(y) * D + 4 * cg) * f;
    }
    if (cg == 0) s_l[rg] = l;
    *reinterpret_cast<f32x4*>(&s_o[rg][4 * cg]) = acc;
    __syncthreads();
    if (rg) return;
    l = 0.f;
    acc = zero4();
#pragma unroll
    for (int y = 0; y < RG; ++y) {
        l += s_l[y];
        acc += *reinterpret_cast<const f32x4*>(&s_o[y][4 * cg]);
    }
    const int rr = b.r0 + row;
    const size_t at = (size_t)(b.t0 + rr / p.G) * p.Hq + hk * p.G + rr % p.G;
    store4(static_cast<T*>(p.out) + at * D + 4 * cg, acc * (l == 0.f ? 0.f : 1.f / l));
    if (p.lse && cg == 0) p.lse[at] = (m + log2f(l)) * LN2;
}

template <class K, class... P> hipError_t launch(K kern, size_t x, size_t lds, hipStream_t st, const P&... p) {
    if (x * 256 > 0xffffffffu) return hipErrorInvalidConfiguration;
    if (lds > 65536) {
        const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kern, dim3((unsigned)x), dim3(256), lds, st, p...);
    return hipGetLastError();
}

// Row tiles of a workgroup: as many as the longest run of rows that a sequence can
// have fills (a packed batch: its mean).
int row_waves(int T, int N, int G, bool packed) {
    const long rows = packed ? ((long)T + N - 1) / N * G : (long)T * G;
    return rows <= 32 ? 1 : rows <= 64 ? 2 : 4;
}

struct Plan {
    int RW;
    long blocks;
    bool shared;
};
Plan make_plan(int T, int N, int Hkv, int G, bool packed) {
    Plan pl;
    pl.RW = row_waves(T, N, G, packed);
    pl.blocks = row_blocks_bound(T, N, G, 32 * pl.RW, packed);
    pl.shared = pl.blocks <= MAX_BLOCKS && pl.blocks * Hkv < 2048;
    return pl;
}

template <class T, int D, int RW> hipError_t attend(const PagedArgs& a, const Plan& pl) {
    AttnParams p{};
    p.q = a.q; p.Kp = a.Kp; p.Vp = a.Vp; p.ctx = a.ctx; p.tree = a.tree; p.out = a.out; p.lse = a.lse;
    p.pages = make_pages(a);
    p.map = SeqMap{a.cu_seqlens, a.T, a.N};
    p.Hq = a.Hq; p.Hkv = a.Hkv; p.G = a.Hq / a.Hkv; p.words = a.words;
    p.capacity = std::min((long)a.width * a.page_size, 0x7ffff000L);
    p.scale = a.scale;
    p.blocks = (int)pl.blocks;
    const size_t items = (size_t)pl.blocks * a.Hkv;
    if (pl.shared) {
        p.wgs = WGS;
        char* ws = static_cast<char*>(a.workspace);
        p.span = reinterpret_cast<int2*>(ws);
        ws += al256(items * 8);
        p.pml = reinterpret_cast<float*>(ws);
        ws += al256((size_t)2 * WGS * 32 * RW * 8);
        p.po = reinterpret_cast<float*>(ws);
    }
    const hipError_t e = launch(paged_attn_kernel<T, D, RW>, pl.shared ? WGS : items, attn_lds<T, D, RW>(), a.stream, p);
    if (e != hipSuccess || !pl.shared) return e;
    return launch(paged_join_kernel<T, D, RW>, items * 32 * RW, 0, a.stream, p);
}

template <class T, int D> hipError_t attend(const PagedArgs& a) {
    const Plan pl = make_plan(a.T, a.N, a.Hkv, a.Hq / a.Hkv, a.cu_seqlens != nullptr);
    return pl.RW == 1 ? attend<T, D, 1>(a, pl) : pl.RW == 2 ? attend<T, D, 2>(a, pl) : attend<T, D, 4>(a, pl);
}

template <class T, int D> hipError_t append(const PagedArgs& a) {
    AppendParams p{};
    p.q = a.q; p.k = a.k; p.v = a.v; p.q_out = a.out; p.Kp = a.Kw; p.Vp = a.Vw;
    p.pos = a.pos; p.ctx = a.ctx; p.freqs = a.freqs;
    p.pages = make_pages(a);
    p.map = SeqMap{a.cu_seqlens, a.T, a.N};
    p.rows = a.cu_seqlens ? a.T : a.N * a.T;
    p.Hq = a.Hq; p.Hkv = a.Hkv; p.rot = a.rot_dim;
    return launch(paged_append_kernel<T, D>, (size_t)(p.rows + 3) / 4, 0, a.stream, p, a.neighbours);
}

#define KDA_PAGED_DIM(d, D, ...)                                       \
    [&] {                                                              \
        switch (d) {                                                   \
            case 32: { constexpr int D = 32; return __VA_ARGS__(); }   \
            case 64: { constexpr int D = 64; return __VA_ARGS__(); }   \
            default: { constexpr int D = 128; return __VA_ARGS__(); }  \
        }                                                              \
    }()

}  // namespace

bool paged_attn_fits(int T, int N, int Hq, int Hkv, bool packed) {
    const Plan pl = make_plan(T, N, Hkv, Hq / Hkv, packed);
    return pl.shared ? pl.blocks * Hkv * 32 * pl.RW < (1 << 24) : pl.blocks * Hkv < (1 << 24);
}

size_t paged_attn_workspace_bytes(int T, int N, int Hq, int Hkv, int d, bool packed) {
    const Plan pl = make_plan(T, N, Hkv, Hq / Hkv, packed);
    if (!pl.shared) return 256;
    const size_t slots = (size_t)2 * WGS * 32 * pl.RW;
    return al256((size_t)pl.blocks * Hkv * 8) + al256(slots * 8) + slots * d * 4 + 256;
}

hipError_t launch_paged_append(const PagedArgs& a) {
    return KDA_PAGED_DIM(a.d, D, [&] { return a.bf16 ? append<uint16_t, D>(a) : append<float, D>(a); });
}
hipError_t launch_paged_attn(const PagedArgs& a) {
    return KDA_PAGED_DIM(a.d, D, [&] { return a.bf16 ? attend<uint16_t, D>(a) : attend<float, D>(a); });
}

}  // namespace kda
