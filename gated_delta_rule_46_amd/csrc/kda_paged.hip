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
#include "kda_bounds.h"
#include "kda_launch.h"

namespace kda {

namespace {

size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

// over the four lanes that hold one column of a 16x16 result
__device__ __forceinline__ float group_max(float v) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return swap_max(fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1])));
}
__device__ __forceinline__ float group_sum(float v) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return swap_sum(__uint_as_float(a[0]) + __uint_as_float(a[1]));
}

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
// are exact, their product is at positions where 32 bits have no fraction left),
// the rest is fp32, rounded once. Bound by memory: 7,213 tokens of eight prompts,
// 16 and 4 heads of 128 channels, bf16 16.4 us at 5.4 TB/s; 46 drafted tokens 4.3 us,
// most of it the way from the offsets over the table to the rows.
template <class T, int D> __global__ void __launch_bounds__(256) paged_append_kernel(AppendParams p, bool neighbours) {
    lds_poison(0);
    __shared__ float s_cos[4][64], s_sin[4][64];
    constexpr int V = 16 / (int)sizeof(T), U = D / (2 * V);   // elements of a piece, units of two of them in a row
    const int w = threadIdx.x / WAVE, lane = threadIdx.x % WAVE;
    // (a wave goes on to further tokens only where a launch has no room for a wave each, from 2^26 on)
    for (long at = (long)blockIdx.x * 4 + w; at < p.rows; at += 4L * gridDim.x) {
        const int t = (int)at;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // the last token's angles are done with
        __builtin_amdgcn_wave_barrier();
        int seq, i;
        if (!token_place(p.map, t, seq, i)) continue;
        const int ctx = p.ctx[seq];
        const long row = (long)ctx + i;
        const int slot = ctx < 0 || row > 0x7fffffffL ? -1 : p.pages.row(seq, (int)row);
        const int half = p.rot / 2;
        if (lane < half) {
            const double turns = (double)(p.pos ? p.pos[t] : row) * (double)p.freqs[lane] * 0.15915494309189535;
            // half turns as two floats: with one, cosines and sines are off by up to 1.9 x 2^-24, with
            // both by 1.3 (no change in time)
            const double x = 2.0 * (turns - rint(turns));
            const float hi = (float)x, lo = (float)(x - (double)hi) * 3.14159265f;
            float sn, cs;
            sincospif(hi, &sn, &cs);
            s_cos[w][lane] = fmaf(-lo, sn, cs);
            s_sin[w][lane] = fmaf(lo, cs, sn);
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
    int HW, groups;         // kv heads that a workgroup takes together, and such groups
    long capacity;          // of a sequence's pages
    float scale;
    int blocks;             // blocks of rows over all sequences
    int wgs;                // workgroups that share the keys, or 0: one for each item
    int2* span;             // [item]: the first and last workgroup of an item that is shared
    float *po, *pml;        // parts: [2 * wgs][HW][R][D], [2 * wgs][HW][R][2]
};

constexpr int MAX_BLOCKS = 1024;   // of a call whose keys are shared out

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
// keys that a block's rows may see, of a sequence with ctx tokens before the new ones
__device__ __forceinline__ int keys_of(const AttnParams& p, const RowBlock& b, int ctx, int R) {
    if (ctx < 0) return 0;
    return (int)min((long)ctx + (p.tree ? b.n : min(b.n, (b.r0 + R - 1) / p.G + 1)), p.capacity);
}

// What a workgroup takes: units (KB keys of one item, a block and a group of kv heads)
// [u, end), counted over the blocks, then the groups; unit u is number it0 of item (v, hg).
// total: of all. Contexts are only known on the device: every workgroup counts all blocks'
// units for itself (2 us at 64 sequences), in place of a launch that does it once.
struct Work {
    long u, end, total;
    int v, hg, it0, wgs, wg;
    bool known;      // b and ctx are those of v
    RowBlock b;
    int ctx;
    // the workgroup that has a unit
    __device__ __forceinline__ int owner(long x) const { return (int)(((x + 1) * wgs - 1) / total); }
};
// LEAST: units that a workgroup has at least, where there are as many. REMAP: workgroups
// that follow each other in the order of units on one die. False for one without work. lds:
// 2 MAX_BLOCKS + 1 words, free again behind the next barrier.
template <int R, int KB, int LEAST, int NT, bool REMAP> __device__ __forceinline__ bool find_work(const AttnParams& p, int* lds, Work& k) {
    const int tid = threadIdx.x, lane = tid % WAVE, w = tid / WAVE;
    k.known = false;
    if (!p.wgs) {
        k.wg = REMAP ? xcd_remap(blockIdx.x, gridDim.x) : (int)blockIdx.x;
        k.u = 0;
        k.end = k.total = k.wgs = 1;
        k.hg = k.wg / p.blocks;
        k.v = k.wg % p.blocks;
        k.it0 = 0;
        return true;
    }
    __shared__ int s_wave[NT / WAVE], s_at[2];
    // offsets and contexts at once, in place of a search through memory (a call has no more
    // sequences than blocks)
    int* const s_ctx = lds;
    int* const s_cu = lds + MAX_BLOCKS;
    for (int i = tid; i < p.map.N; i += NT) s_ctx[i] = p.ctx[i];
    if (p.map.cu)
        for (int i = tid; i <= p.map.N; i += NT) s_cu[i] = p.map.cu[i];
    __syncthreads();
    const SeqMap map{p.map.cu ? s_cu : nullptr, p.map.T, p.map.N};
    const int each = (p.blocks + NT - 1) / NT, b0 = tid * each;   // neighbours that a thread counts
    constexpr int MOST = (MAX_BLOCKS + NT - 1) / NT;
    int mine[MOST], sum = 0;
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
        RowBlock rb;
        mine[i] = 0;
        if (i < each && b0 + i < p.blocks && row_block(map, p.G, R, b0 + i, rb))
            mine[i] = max((keys_of(p, rb, s_ctx[rb.seq], R) + KB - 1) / KB, 1);
        sum += mine[i];
    }
    int before = sum;
#pragma unroll
    for (int o = 1; o < WAVE; o *= 2) {
        const int y = __shfl_up(before, o, WAVE);
        if (lane >= o) before += y;
    }
    if (lane == 63) s_wave[w] = before;
    __syncthreads();
    before -= sum;
    int of_head = 0;
#pragma unroll
    for (int i = 0; i < NT / WAVE; ++i) {
        before += i < w ? s_wave[i] : 0;
        of_head += s_wave[i];
    }
    of_head = __builtin_amdgcn_readfirstlane(of_head);
    k.total = (long)of_head * p.groups;
    k.wgs = (int)min((long)p.wgs, (k.total + LEAST - 1) / LEAST);
    if ((int)blockIdx.x >= k.wgs) return false;
    k.wg = REMAP ? xcd_remap(blockIdx.x, k.wgs) : (int)blockIdx.x;
    k.u = k.total * k.wg / k.wgs;
    k.end = k.total * (k.wg + 1) / k.wgs;
    k.hg = (int)(k.u / of_head);
    const int at = (int)(k.u - (long)k.hg * of_head);
#pragma unroll
    for (int i = 0; i < MOST; ++i) {   // one block of one thread holds the unit
        if (at >= before && at < before + mine[i]) {
            s_at[0] = b0 + i;
            s_at[1] = at - before;
        }
        before += mine[i];
    }
    __syncthreads();
    k.v = __builtin_amdgcn_readfirstlane(s_at[0]);
    k.it0 = __builtin_amdgcn_readfirstlane(s_at[1]);
    row_block(map, p.G, R, k.v, k.b);
    k.b = RowBlock{__builtin_amdgcn_readfirstlane(k.b.seq), __builtin_amdgcn_readfirstlane(k.b.r0),
                   __builtin_amdgcn_readfirstlane(k.b.rows), __builtin_amdgcn_readfirstlane(k.b.n),
                   (long)__builtin_amdgcn_readfirstlane((int)k.b.t0)};   // (tokens over the batch: 31 bits)
    k.ctx = __builtin_amdgcn_readfirstlane(s_ctx[k.b.seq]);
    k.known = true;
    return true;
}

// The new tokens that one row sees, as bits.
struct Seen {
    const int32_t* bits;   // the token's words, or null: every token up to `tok`
    int words, ctx, tok;
    // of the 32 keys from j0 on
    __device__ __forceinline__ uint32_t operator()(int j0) const {
        const int d = j0 - ctx;   // among the new tokens
        if (bits == nullptr) {
            // (a context may be any number: tok - d without a sign)
            const uint32_t m = tok >= d ? min((uint32_t)tok - (uint32_t)d, 31u) + 1u : 0u;
            return m == 32 ? ~0u : (1u << m) - 1u;
        }
        if (d <= -32) return ~0u;
        if (d < 0) return ((1u << -d) - 1u) | (uint32_t)bits[0] << -d;
        const int at = d >> 5, sh = d & 31;
        const uint32_t x = at < words ? (uint32_t)bits[at] : 0u;
        const uint32_t y = sh && at + 1 < words ? (uint32_t)bits[at + 1] << (32 - sh) : 0u;
        return x >> sh | y;
    }
};

// Strides of tiles of values, which only transposing reads touch. Those of a 16x16 product
// take 16 rows of 8 dwords, those of a 32x32 product 8 rows of 16: rows 8 (16) dwords apart
// cover the 64 banks evenly, while at tile_stride's 4, which suits reads along rows, they
// met (half of all LDS cycles of 2,048 rows over 6,144 tokens). fp32 reads single elements.
template <class T> constexpr int v_stride16(int d) { return sizeof(T) == 2 ? d + 16 : tile_stride<T>(d); }
template <class T> constexpr int v_stride32(int d) { return sizeof(T) == 2 ? (d == 32 ? 32 : d + 32) : tile_stride<T>(d); }

// ---------------------------------------------------------------- few rows

// Up to 16 RT rows a block, tiles of 16x16 and 32 deep. A wave has one kv head and tiles
// of 32 keys of its own; the waves of a workgroup take HW heads of the same keys, which lie
// side by side in memory, and every KS-th tile where there are fewer heads than waves. Keys
// go from memory to the operand as they lie (a lane has 8 values of one key), values through
// the wave's own LDS for the transposing read; the next DEPTH tiles' loads are under way
// while a tile is worked on. A lane owns one row of the scores, whose layout is the next
// product's operand (kpos order). bf16 probabilities enter it as two bf16 numbers (3 of 40 us
// at 8 sequences of 8,192 tokens): o is then off by no more than its own rounding.
// Bound by memory: one token of 64 sequences of 100 to 4,096 tokens, 32 and 8 heads of 128
// channels, bf16 112 us at 5.0 TB/s, of 4,096 tokens each 197 us at 5.5. Small calls: 13 us
// for 2,048 to 8,192 tokens of one sequence, of which 2 are the plan's, 2 to 4 the loads' way
// and 2 to 4 the join of the waves' shares. Two tiles ahead with 32 rows spill (89 us, one 49);
// with 16 at 128 channels bf16 three registers wait in scratch from before the loop over tiles
// until behind it, none within.
template <class T, int D, int RT> struct Few {
    // workgroups of eight waves, two a SIMD, or of four where registers leave room for one
    static constexpr int NW = sizeof(T) == 4 && D == 128 ? 4 : 8, DEPTH = RT == 1 ? 2 : 1, R = 16 * RT;
    static constexpr size_t tiles = sizeof(T) * NW * 32 * v_stride16<T>(D), join = sizeof(float) * NW * R * (D + 4);
    static constexpr size_t lds = tiles > join ? tiles : join;
};

template <class T, int D, int RT>
__global__ void __launch_bounds__((64 * Few<T, D, RT>::NW), (Few<T, D, RT>::NW / 4)) paged_few_kernel(AttnParams p) {
    using F = Few<T, D, RT>;
    constexpr int NW = F::NW, NT = 64 * NW, DEPTH = F::DEPTH, R = F::R, KB = 32;
    constexpr int ST = v_stride16<T>(D), KD = D / 32, MD = D / 16, JS = D + 4;
    constexpr int PER = 16 / (int)sizeof(T), CPR = D / PER, NL = 32 * CPR / 64;
    using V8 = typename Frag<T>::V;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float s_top[NW][R], s_sum[NW][R];
    lds_poison((uint32_t)F::lds);
    const int tid = threadIdx.x, lane = tid % WAVE, w = wave_id(), n = lane & 15, g = lane >> 4;
    T* const tv = reinterpret_cast<T*>(smem) + (size_t)w * 32 * ST;
    const float c = p.scale * LOG2E;
    const size_t rs = (size_t)p.Hkv * D;
    Work k;
    const int HW = p.HW, KS = NW / HW, wh = w % HW, wk = w / HW;
    if (!find_work<R, KB, 2, NT, false>(p, reinterpret_cast<int*>(smem), k)) return;

    for (long u = k.u; u < k.end && k.hg < p.groups; k.it0 = 0) {
        RowBlock b = k.b;
        if (!k.known && !row_block(p.map, p.G, R, k.v, b)) {   // an empty number of a packed batch
            if (!p.wgs) return;
            if (++k.v == p.blocks) {
                k.v = 0;
                ++k.hg;
            }
            continue;
        }
        const int ctx = k.known ? k.ctx : p.ctx[b.seq], keys = keys_of(p, b, ctx, R);
        k.known = false;
        const int units = max((keys + KB - 1) / KB, 1), it0 = k.it0;
        const int it1 = p.wgs ? (int)min((long)units, it0 + (k.end - u)) : units;
        const bool whole = it0 == 0 && it1 == units;
        const int rows = min(b.rows - b.r0, R);
        const int hk = k.hg * HW + wh;
        const T* const K = static_cast<const T*>(p.Kp) + (size_t)hk * D;
        const T* const V = static_cast<const T*>(p.Vp) + (size_t)hk * D;
        // row of the block -> its place in q, o
        auto q_row = [&](int r, int head) {
            const int rr = b.r0 + r;
            return (size_t)(b.t0 + rr / p.G) * p.Hq + head * p.G + rr % p.G;
        };
        Seen seen[RT];
        V8 qf[RT][KD];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const int r = 16 * t + n;
            const bool live = r < rows;
            const int tok = (b.r0 + (live ? r : 0)) / p.G;
            seen[t] = Seen{p.tree ? p.tree + (size_t)(b.t0 + tok) * p.words : nullptr, p.words, ctx, tok};
#pragma unroll
            for (int ks = 0; ks < KD; ++ks)
                qf[t][ks] = load8<T>(static_cast<const T*>(p.q) + q_row(live ? r : 0, hk) * D + 32 * ks + 8 * g, live);
        }
        // row in the cache of key (tile's first + lane), or -1
        auto lookup = [&](int it) {
            const int j = it * KB + lane;
            return it < it1 && lane < 32 && j < keys ? p.pages.row(b.seq, j) : -1;
        };
        V8 kf[DEPTH][2][KD];
        u32x4 rv[DEPTH][NL];
        auto fetch_k = [&](auto d, int where) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const T* const src = K + (size_t)max(__shfl(where, 16 * x + n, WAVE), 0) * rs + 8 * g;
#pragma unroll
                for (int ks = 0; ks < KD; ++ks) kf[d.value][x][ks] = load8<T>(src + 32 * ks, true);
            }
        };
        auto fetch_v = [&](auto d, int where) {
#pragma unroll
            for (int m = 0; m < NL; ++m) {
                const int e = lane + 64 * m;
                rv[d.value][m] = *reinterpret_cast<const u32x4*>(V + (size_t)max(__shfl(where, e / CPR, WAVE), 0) * rs + e % CPR * PER);
            }
        };
        f32x4 O[RT][MD];
        float top[RT], sum[RT];   // sum: this lane's quarter of the keys
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            top[t] = -INFINITY;
            sum[t] = 0.f;
#pragma unroll
            for (int m = 0; m < MD; ++m) O[t][m] = zero4();
        }
        int where[DEPTH], next[DEPTH];   // rows of the tiles under way, and of those behind them
        auto each = [](auto f) {
            f(std::integral_constant<int, 0>());
            if constexpr (DEPTH > 1) f(std::integral_constant<int, DEPTH - 1>());
        };
        each([&](auto d) { where[d.value] = lookup(it0 + wk + d.value * KS); });
        __syncthreads();   // the last item's join is done with
        each([&](auto d) {
            fetch_k(d, where[d.value]);
            fetch_v(d, where[d.value]);
        });
        each([&](auto d) { next[d.value] = lookup(it0 + wk + (DEPTH + d.value) * KS); });
        auto tile = [&](auto d, int it) {
            const int j0 = it * KB;
            const uint32_t held = (uint32_t)__ballot(where[d.value] >= 0);
            const bool more = it + DEPTH * KS < it1;
            f32x4 s[RT][2];
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    s[t][x] = zero4();
#pragma unroll
                    for (int ks = 0; ks < KD; ++ks) s[t][x] = mma(kf[d.value][x][ks], qf[t][ks], s[t][x]);
                }
            if (more) fetch_k(d, next[d.value]);
#pragma unroll
            for (int m = 0; m < NL; ++m) {
                const int e = lane + 64 * m, row = e / CPR;
                if (held != ~0u && !(held >> row & 1u)) rv[d.value][m] = u32x4{0u, 0u, 0u, 0u};   // not this sequence's
                *reinterpret_cast<u32x4*>(tv + row * ST + e % CPR * PER) = rv[d.value][m];
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // the tile is this wave's own
            __builtin_amdgcn_wave_barrier();
            if (more) fetch_v(d, next[d.value]);
            where[d.value] = next[d.value];
            next[d.value] = lookup(it + 2 * DEPTH * KS);
            const bool all = held == ~0u && j0 + 31 - (p.tree ? -1 : b.r0 / p.G) <= ctx;   // every row sees every key
            bf16pair pb[RT];
            f32x8 pf[RT];
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const uint32_t see = all ? ~0u : (seen[t](j0) & held) >> 4 * g;
                float mt = -INFINITY;
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        s[t][x][r] = see >> (16 * x + r) & 1u ? s[t][x][r] * c : -INFINITY;
                        mt = __builtin_elementwise_maximum(mt, s[t][x][r]);
                    }
                mt = group_max(mt);
                const float next_top = fmaxf(top[t], mt);
                const float base = next_top == -INFINITY ? 0.f : next_top;
                const float down = fast_exp2(top[t] - base);
                top[t] = next_top;
                sum[t] *= down;
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        pf[t][4 * x + r] = fast_exp2(s[t][x][r] - base);
                        sum[t] += pf[t][4 * x + r];
                    }
                if constexpr (sizeof(T) == 2) pb[t] = split8(pf[t]);
#pragma unroll
                for (int m = 0; m < MD; ++m) O[t][m] *= down;
            }
#pragma unroll
            for (int m = 0; m < MD; ++m) {
                const V8 vf = frag_tr(tv, ST, 0, 16 * m, g, n);
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    if constexpr (sizeof(T) == 2) O[t][m] = mma(vf, pb[t].lo, mma(vf, pb[t].hi, O[t][m]));
                    else O[t][m] = mma(vf, pf[t], O[t][m]);
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        };
        for (int i = it0; i < it1; i += DEPTH * KS) {
            const int it = i + wk;
            each([&](auto d) {
                if (it + d.value * KS < it1) tile(d, it + d.value * KS);
            });
            // Keeps the waves on the same rows; without it the oldest ones run ahead and end early
            // (64 sequences of 4,096 tokens, 8 kv heads: 200 against 197 us). With one tile ahead
            // it costs more than that (8 times 8 tokens over 8,192: 47 against 49).
            if constexpr (DEPTH > 1) __builtin_amdgcn_s_barrier();
        }
        float probe = 0.f;
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            sum[t] = group_sum(sum[t]);
#pragma unroll
            for (int m = 0; m < MD; ++m) probe += (O[t][m][0] + O[t][m][1]) * 0.f + (O[t][m][2] + O[t][m][3]) * 0.f;
        }
        // An Inf or NaN in v at a key that a tile holds but a row does not see has entered
        // that row as 0 * v. Then o is formed again, one key at a time, from what each row sees.
        if (__any(probe != 0.f)) {
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const bool live = 16 * t + n < rows;
                const T* const q = static_cast<const T*>(p.q) + q_row(live ? 16 * t + n : 0, hk) * D;
                const float base = top[t] == -INFINITY ? 0.f : top[t];
#pragma unroll
                for (int m = 0; m < MD; ++m) O[t][m] = zero4();
                for (int it = it0 + wk; it < it1; it += KS) {
                    const int at32 = lookup(it);
                    for (int j = 0; j < 32; ++j) {
                        const int at = __shfl(at32, j, WAVE);
                        const bool in = live && at >= 0 && (seen[t](it * KB) >> j & 1u);
                        if (!__any(in)) continue;
                        const T* const kr = K + (size_t)max(at, 0) * rs;
                        const T* const vr = V + (size_t)max(at, 0) * rs + 4 * g;
                        float dot = 0.f;
                        for (int x = 0; x < D; x += 8) {
                            const f32x8 y = widen(load8<T>(q + x, true)) * widen(load8<T>(kr + x, true));
                            dot += ((y[0] + y[1]) + (y[2] + y[3])) + ((y[4] + y[5]) + (y[6] + y[7]));
                        }
                        const float e = fast_exp2(dot * c - base);
                        if (!in) continue;
#pragma unroll
                        for (int m = 0; m < MD; ++m)
#pragma unroll
                            for (int r = 0; r < 4; ++r) O[t][m][r] += e * from_el(vr[16 * m + r]);
                    }
                }
            }
        }
        // the waves' shares, joined through LDS in the tiles' place: [wave][row][D]
        float* const so = reinterpret_cast<float*>(smem);
        __syncthreads();
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            if (g == 0) {
                s_top[w][16 * t + n] = top[t];
                s_sum[w][16 * t + n] = sum[t];
            }
            if (16 * t + n < rows) {
#pragma unroll
                for (int m = 0; m < MD; ++m) *reinterpret_cast<f32x4*>(so + (size_t)(w * R + 16 * t + n) * JS + 16 * m + 4 * g) = O[t][m];
            }
        }
        __syncthreads();
        for (int x = tid; x < HW * rows * (D / 4); x += NT) {
            const int d = x % (D / 4) * 4, hr = x / (D / 4), h = hr / rows, r = hr - h * rows;
            float m = -INFINITY, l = 0.f;
            for (int y = h; y < NW; y += HW) m = fmaxf(m, s_top[y][r]);
            const float base = m == -INFINITY ? 0.f : m;
            f32x4 acc = zero4();
            for (int y = h; y < NW; y += HW) {
                const float f = fast_exp2(s_top[y][r] - base);
                l += f * s_sum[y][r];
                acc += *reinterpret_cast<const f32x4*>(so + (size_t)(y * R + r) * JS + d) * f;
            }
            if (whole) {
                const size_t at = q_row(r, k.hg * HW + h);
                store4(static_cast<T*>(p.out) + at * D + d, acc * (l == 0.f ? 0.f : 1.f / l));
                if (p.lse && d == 0) p.lse[at] = (m + log2f(l)) * LN2;
            } else {
                const size_t slot = (((size_t)2 * k.wg + (it0 == 0 ? 1 : 0)) * HW + h) * R + r;
                *reinterpret_cast<f32x4*>(p.po + slot * D + d) = acc;
                if (d == 0) {
                    p.pml[2 * slot] = m;
                    p.pml[2 * slot + 1] = l;
                }
            }
        }
        if (p.wgs && it0 == 0 && tid == 0)
            p.span[k.v * p.groups + k.hg] = make_int2(k.wg, k.owner(u + units - 1));
        u += it1 - it0;
        if (++k.v == p.blocks) {
            k.v = 0;
            ++k.hg;
        }
    }
}

// ---------------------------------------------------------------- more rows

// Scores and o of 32 rows a wave on 32x32 tiles: rows stay in registers (a lane owns one),
// keys and values come through LDS, twice over, for the RW waves that share them. RW: rows'
// tiles of 32 a workgroup has; KS = 4 / RW groups of waves take every KS-th tile of keys each.
// bf16 probabilities enter the second product as two bf16 numbers here too, so that a token is
// as exact in a block of many rows as in one of few. Rounded once, for a single product, they
// put o off by 1.4 times its own rounding (2,048 tokens over 6,144 168 us, two products 206;
// 2,048 alone 51 and 56; 8 trees of 64 90 and 100). Bound by the turns that scores,
// exponentials and products take within two waves a SIMD: 2,048 tokens over 6,144, 16 and 4
// heads of 128 channels, bf16 206 to 216 us (560 to 590 TFLOP/s), matrix units busy for 40% of
// it. Without gain, tried with one product: 256 rows in eight waves (3 to 6% faster from 2,048
// rows and long contexts on, 3 to 5% slower at 256 rows and for short ones), with its two halves
// of waves a phase apart as well (189 us against 175), two tiles of rows a wave at one wave a SIMD
// (213), exponentials beside the next tile's scores (207), wave priorities and orders of the loads.
template <class T, int RW> struct Shape {
    static constexpr int KS = 4 / RW, R = 32 * RW, KT = sizeof(T) == 2 && RW == 4 ? 64 : 32, KB = KS * KT;
};
template <class T, int D, int RW> constexpr size_t rows_lds() {
    using S = Shape<T, RW>;
    const size_t tiles = sizeof(T) * S::KS * 2 * S::KT * (tile_stride<T>(D) + v_stride32<T>(D));
    const size_t join = S::KS > 1 ? sizeof(float) * 4 * 64 * (16 * (D / 32) + 2) : 0;
    return std::max(tiles, join);
}

// Half b of a tile of probabilities as operands: fp32 as they are, bf16 as two numbers, the
// upper half of p's bits and the rest rounded (together off by 2^-15 at most; a NaN of the
// arithmetic stays one). To round the first as well costs 1 to 2% more.
template <class T> struct Weights {
    typename Frag<T>::V hi;
    __device__ __forceinline__ Weights(const f32x16& x, int b) : hi(rows16<T>(x, b)) {}
};
template <> struct Weights<uint16_t> {
    bf16x8 hi, lo;
    __device__ __forceinline__ Weights(const f32x16& x, int b) {
        u32x4 top;
        f32x8 rest;
#pragma unroll
        for (int m = 0; m < 8; m += 2) {
            const uint32_t y = __float_as_uint(x[8 * b + m]), z = __float_as_uint(x[8 * b + m + 1]);
            top[m / 2] = __builtin_amdgcn_perm(z, y, 0x07060302u);
            rest[m] = x[8 * b + m] - __uint_as_float(y & 0xffff0000u);
            rest[m + 1] = x[8 * b + m + 1] - __uint_as_float(z & 0xffff0000u);
        }
        hi = __builtin_bit_cast(bf16x8, top);
        lo = narrow<uint16_t>(rest);
    }
};

// workgroups that a CU holds at once
template <class T, int D, int RW> constexpr int rows_at_once() { return rows_lds<T, D, RW>() > 80 * 1024 ? 1 : 2; }

template <class T, int D, int RW> __global__ void __launch_bounds__(256, (rows_at_once<T, D, RW>())) paged_rows_kernel(AttnParams p) {
    using S = Shape<T, RW>;
    constexpr int KS = S::KS, R = S::R, KT = S::KT, KB = S::KB, NX = KT / 32, GT = 64 * RW;
    constexpr int ST = tile_stride<T>(D), SV = v_stride32<T>(D), KD = D / 16, MD = D / 32, PER = 16 / (int)sizeof(T), CPR = D / PER, NL = KT * CPR / GT;
    using V8 = typename Frag<T>::V;
    extern __shared__ __align__(16) unsigned char smem[];
    lds_poison((uint32_t)rows_lds<T, D, RW>());
    const int tid = threadIdx.x, lane = tid % WAVE, w = wave_id(), n = lane & 31, h2 = lane >> 5;
    const int wr = w % RW, wk = w / RW, gt = tid - wk * GT;
    T* const tiles = reinterpret_cast<T*>(smem) + (size_t)wk * 2 * KT * (ST + SV);   // [buffer][k [KT][ST], v [KT][SV]]
    // the scale's sign goes into q, exactly, and so does a scale of zero: maxima scale as they stand
    const float c = p.scale == 0.f ? 1.f : fabsf(p.scale) * LOG2E;
    const size_t rs = (size_t)p.Hkv * D;
    const bool chunks = p.pages.page % (GT / CPR) == 0;
    // this thread's places in a tile: of what it brings, and of its operands
    const int put_k = gt / CPR * ST + gt % CPR * PER, put_v = gt / CPR * SV + gt % CPR * PER;
    const int at_k = n * ST + 8 * h2;
    const int at_v = sizeof(T) == 2 ? (4 * h2 + ((lane & 15) >> 2)) * SV + (lane & 16) + 4 * (lane & 3) : 4 * h2 * SV + n;

    Work k;
    if (!find_work<R, KB, 1, 256, true>(p, reinterpret_cast<int*>(smem), k)) return;
    long u = k.u;
    const long end = k.end;
    int v = k.v, hk = k.hg, it0 = k.it0;

    for (; u < end && hk < p.Hkv; it0 = 0) {
        RowBlock b = k.b;
        if (!k.known && !row_block(p.map, p.G, R, v, b)) {   // an empty number of a packed batch
            if (!p.wgs) return;
            if (++v == p.blocks) {
                v = 0;
                ++hk;
            }
            continue;
        }
        const int ctx = k.known ? k.ctx : p.ctx[b.seq], keys = keys_of(p, b, ctx, R);
        k.known = false;
        const int units = max((keys + KB - 1) / KB, 1);
        const int it1 = p.wgs ? (int)min((long)units, it0 + (end - u)) : units;
        const bool whole = it0 == 0 && it1 == units;
        // this lane's row; formed where it is needed, so that no register holds it over the loop
        struct Row {
            bool live;
            int tok;
            size_t at;   // its place in q, o
        };
        auto row_of = [&](int n) {
            const int rr = b.r0 + 32 * wr + n;
            const bool live = rr < b.rows;
            const int tok = (live ? rr : 0) / p.G, head = hk * p.G + (live ? rr : 0) % p.G;
            return Row{live, tok, (size_t)(b.t0 + tok) * p.Hq + head};
        };

        V8 qf[KD];
        {
            const Row row = row_of(n);
#pragma unroll
            for (int ks = 0; ks < KD; ++ks) {
                qf[ks] = load8<T>(static_cast<const T*>(p.q) + row.at * D + 8 * h2 + 16 * ks, row.live);
                if (p.scale <= 0.f) qf[ks] = p.scale < 0.f ? -qf[ks] : narrow<T>(widen(qf[ks]) * 0.f);
            }
        }
        const T* const K = static_cast<const T*>(p.Kp) + (size_t)hk * D;
        const T* const V = static_cast<const T*>(p.Vp) + (size_t)hk * D;

        // the row in the cache of key (tile's first + lane), or -1
        auto lookup = [&](int it) {
            const int j = (it * KS + wk) * KT + lane;
            return lane < KT && j < keys ? p.pages.row(b.seq, j) : -1;
        };
        u32x4 rk[NL], rv[NL];
        // Pages of whole chunks (the rows that one load of the group's threads covers) have one
        // address a chunk, the same in every lane; others an address for each row.
        auto fetch = [&](int where) {
            const int here_gt = here(gt);
            if (chunks) {
                const uint32_t off = (uint32_t)(here_gt / CPR) * (uint32_t)rs + (uint32_t)(here_gt % CPR * PER);
#pragma unroll
                for (int m = 0; m < NL; ++m) {
                    const size_t at = (size_t)max(__builtin_amdgcn_readlane(where, m * (GT / CPR)), 0) * rs;
                    rk[m] = *reinterpret_cast<const u32x4*>(K + at + off);
                    rv[m] = *reinterpret_cast<const u32x4*>(V + at + off);
                }
                return;
            }
#pragma unroll
            for (int m = 0; m < NL; ++m) {
                const int e = here_gt + m * GT, at = max(__shfl(where, e / CPR, WAVE), 0);
                const size_t o = (size_t)at * rs + e % CPR * PER;
                rk[m] = *reinterpret_cast<const u32x4*>(K + o);
                rv[m] = *reinterpret_cast<const u32x4*>(V + o);
            }
        };
        // (rows that are not this sequence's become zeros)
        auto put = [&](T* t, uint64_t held, bool full) {
            T* const tk = t + put_k;
            T* const tv = t + KT * ST + put_v;
            constexpr int RPC = GT / CPR;
            if (full) {
#pragma unroll
                for (int m = 0; m < NL; ++m) {
                    *reinterpret_cast<u32x4*>(tk + m * RPC * ST) = rk[m];
                    *reinterpret_cast<u32x4*>(tv + m * RPC * SV) = rv[m];
                }
                return;
            }
#pragma unroll
            for (int m = 0; m < NL; ++m) {
                const uint32_t keep = held >> (gt / CPR + m * RPC) & 1 ? ~0u : 0u;
                *reinterpret_cast<u32x4*>(tk + m * RPC * ST) = rk[m] & keep;
                *reinterpret_cast<u32x4*>(tv + m * RPC * SV) = rv[m] & keep;
            }
        };
        auto seen_by = [&](int tok) {
            return Seen{p.tree ? p.tree + (size_t)(b.t0 + tok) * p.words : nullptr, p.words, ctx, tok};
        };

        f32x16 O[MD];
#pragma unroll
        for (int m = 0; m < MD; ++m) O[m] = zero16();
        float top = -INFINITY, sum = 0.f;   // sum: this lane's half of the keys

        auto tile = [&](const T* tk, const T* tv, int j0, uint64_t held, bool masked) {
            tk += at_k;
            tv += at_v;
            f32x16 s[NX];
            V8 vf[MD];
#pragma unroll
            for (int x = 0; x < NX; ++x) s[x] = zero16();
            constexpr int HD = KD > 4 ? KD / 2 : KD;   // operands of half the head at a time: registers
#pragma unroll
            for (int k0 = 0; k0 < KD; k0 += HD) {
                V8 kf[NX][HD];
#pragma unroll
                for (int ks = 0; ks < HD; ++ks)
#pragma unroll
                    for (int x = 0; x < NX; ++x) kf[x][ks] = nat32<T>(tk, ST, 32 * x, 16 * (k0 + ks), 0, 0);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int ks = 0; ks < HD; ++ks)
#pragma unroll
                    for (int x = 0; x < NX; ++x) s[x] = mma32(kf[x][ks], qf[k0 + ks], s[x]);
                if (k0 + HD < KD) __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int m = 0; m < MD; ++m) vf[m] = tr32(tv, SV, 0, 32 * m, 0);
            __builtin_amdgcn_sched_barrier(0);
            if (masked) {
                const Seen visible = seen_by(row_of(n).tok);
#pragma unroll
                for (int x = 0; x < NX; ++x) {
                    const uint32_t see = (visible(j0 + 32 * x) & (uint32_t)(held >> 32 * x)) >> 4 * h2;
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[x][r] = see >> result_row(r, 0) & 1u ? s[x][r] : -INFINITY;
                }
            }
            float mt = tree_max(s[0]);
#pragma unroll
            for (int x = 1; x < NX; ++x) mt = __builtin_elementwise_maximum(mt, tree_max(s[x]));
            mt = swap_max(mt * c);
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
            auto weigh = [&](int x) {   // scores of 32 keys to probabilities
                float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    s[x][r] = fast_exp2(fmaf(s[x][r], c, -base));
                    part[r & 3] += s[x][r];
                }
                sum += (part[0] + part[1]) + (part[2] + part[3]);
            };
            weigh(0);
#pragma unroll
            for (int kb = 0; kb < KT / 16; ++kb) {
                V8 next[MD];
                if (kb + 1 < KT / 16) {
#pragma unroll
                    for (int m = 0; m < MD; ++m) next[m] = tr32(tv, SV, 16 * (kb + 1), 32 * m, 0);
                }
                const Weights<T> pf(s[kb / 2], kb % 2);
#pragma unroll
                for (int m = 0; m < MD; ++m) O[m] = mma32(vf[m], pf.hi, O[m]);
                if constexpr (sizeof(T) == 2) {
#pragma unroll
                    for (int m = 0; m < MD; ++m) O[m] = mma32(vf[m], pf.lo, O[m]);
                }
                if (kb % 2 == 0 && kb / 2 + 1 < NX) weigh(kb / 2 + 1);
                if (kb + 1 < KT / 16) {
#pragma unroll
                    for (int m = 0; m < MD; ++m) vf[m] = next[m];
                }
            }
        };

        int where = lookup(it0);
        uint64_t held = __ballot(where >= 0);
        constexpr uint64_t ALL = KT == 64 ? ~0ull : 0xffffffffull;
        __syncthreads();   // the last item's tiles and joins are done with
        fetch(where);
        int where_next = it0 + 1 < it1 ? lookup(it0 + 1) : -1;
        for (int it = it0; it < it1; ++it) {
            T* const t = tiles + (size_t)(it & 1) * KT * (ST + SV);
            put(t, held, held == ALL);
            __syncthreads();
            const uint64_t now = held;
            if (it + 1 < it1) {
                held = __ballot(where_next >= 0);
                fetch(where_next);
                where_next = it + 2 < it1 ? lookup(it + 2) : -1;
            }
            const int j0 = (it * KS + wk) * KT;
            if (now) {
                const int own = p.tree ? -1 : (b.r0 + 32 * wr) / p.G;   // the last new token that every row of this wave sees
                tile(t, t + KT * ST, j0, now, now != ALL || j0 + KT - 1 - own > ctx);
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
        const Row row = row_of(here(n));
        if (__any(row.live && probe != 0.f)) {
            const Seen visible = seen_by(row.tok);
            const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
            for (int m = 0; m < MD; ++m) O[m] = zero16();
            for (int it = it0; it < it1; ++it) {
                const int rows = lookup(it), j0 = (it * KS + wk) * KT;
                for (int j = 0; j < KT; ++j) {
                    const int at = __shfl(rows, j, WAVE);
                    const bool in = row.live && at >= 0 && (visible(j0 + (j & 32)) >> (j & 31) & 1u);
                    if (!__any(in)) continue;
                    const T* const kr = K + (size_t)max(at, 0) * rs;
                    const T* const vr = V + (size_t)max(at, 0) * rs;
                    float dot = 0.f;
                    for (int x = 0; x < D; x += 8) {
                        const f32x8 y = widen(load8<T>(static_cast<const T*>(p.q) + row.at * D + x, true)) * widen(load8<T>(kr + x, true));
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
        if (wk == 0 && row.live) {
            if (whole) {
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                T* out = static_cast<T*>(p.out) + row.at * D;
#pragma unroll
                for (int m = 0; m < MD; ++m) store_tile<T>(out + 32 * m, O[m], inv, h2);
                if (p.lse && h2 == 0) p.lse[row.at] = (top + log2f(sum)) * LN2;
            } else {
                const size_t slot = ((size_t)2 * k.wg + (it0 == 0 ? 1 : 0)) * R + 32 * wr + n;
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
            p.span[v * p.Hkv + hk] = make_int2(k.wg, k.owner(u + units - 1));
        u += it1 - it0;
        if (++v == p.blocks) {
            v = 0;
            ++hk;
        }
    }
}

// Joins the parts of a shared item's rows, four values a thread, in J workgroups: as many
// rows at a time as a workgroup has room for, or (SPREAD) one row at a time with its parts
// spread over the workgroup, for few rows in many parts. Parts are added in their order: the
// same bits every time. 64 sequences 8.1 us, one of 8,191 tokens 4.7, 2,048 rows 14.1 (60 MB).
template <class T, int D, int R, bool SPREAD> __global__ void __launch_bounds__(256) paged_join_kernel(AttnParams p, int J) {
    lds_poison(0);
    constexpr int CG = D / 4, RG = 256 / CG;
    const int at_head = blockIdx.x / J, j = blockIdx.x % J, v = at_head / p.Hkv, hk = at_head % p.Hkv, wh = hk % p.HW;
    RowBlock b;
    if (!row_block(p.map, p.G, R, v, b)) return;
    const int2 span = p.span[v * p.groups + hk / p.HW];
    const int parts = span.y - span.x + 1, tid = threadIdx.x, cg = tid % CG, rg = tid / CG, rows = min(b.rows - b.r0, R);
    if (parts == 1 || !parts_exist(span.x, span.y, p.wgs)) return;
    auto finish = [&](int row, float m, float l, const f32x4& acc) {
        const int rr = b.r0 + row;
        const size_t at = (size_t)(b.t0 + rr / p.G) * p.Hq + hk * p.G + rr % p.G;
        store4(static_cast<T*>(p.out) + at * D + 4 * cg, acc * (l == 0.f ? 0.f : 1.f / l));
        if (p.lse && cg == 0) p.lse[at] = (m + log2f(l)) * LN2;
    };
    auto slot = [&](int y, int row) { return (((size_t)2 * (span.x + y) + (y == 0 ? 1 : 0)) * p.HW + wh) * R + row; };
    // a row's parts y0, y0 + step, ..
    auto collect = [&](int row, int y0, int step, float base, float& l, f32x4& acc) {
        l = 0.f;
        acc = zero4();
#pragma unroll 8
        for (int y = y0; y < parts; y += step) {
            const float2 ml = *reinterpret_cast<const float2*>(p.pml + 2 * slot(y, row));
            const f32x4 o = *reinterpret_cast<const f32x4*>(p.po + slot(y, row) * D + 4 * cg);
            const float f = fast_exp2(ml.x - base);
            l += f * ml.y;
            acc += o * f;
        }
    };
    float l;
    f32x4 acc;
    if constexpr (!SPREAD) {
        for (int row = j * RG + rg; row < rows; row += J * RG) {
            float m = -INFINITY;
#pragma unroll 8
            for (int y = 0; y < parts; ++y) m = fmaxf(m, p.pml[2 * slot(y, row)]);
            collect(row, 0, 1, m == -INFINITY ? 0.f : m, l, acc);
            finish(row, m, l, acc);
        }
        return;
    }
    __shared__ float s_m[4], s_l[RG];
    __shared__ __align__(16) float s_o[RG][D];
    for (int row = j; row < rows; row += J) {
        float m = -INFINITY;
        for (int y = tid; y < parts; y += 256) m = fmaxf(m, p.pml[2 * slot(y, row)]);
#pragma unroll
        for (int o = 32; o; o /= 2) m = fmaxf(m, __shfl_xor(m, o, WAVE));
        __syncthreads();   // the last row's sums are done with
        if (tid % WAVE == 0) s_m[tid / WAVE] = m;
        __syncthreads();
        m = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
        collect(row, rg, RG, m == -INFINITY ? 0.f : m, l, acc);
        if (cg == 0) s_l[rg] = l;
        *reinterpret_cast<f32x4*>(&s_o[rg][4 * cg]) = acc;
        __syncthreads();
        if (rg) continue;
        l = 0.f;
        acc = zero4();
#pragma unroll
        for (int y = 0; y < RG; ++y) {
            l += s_l[y];
            acc += *reinterpret_cast<const f32x4*>(&s_o[y][4 * cg]);
        }
        finish(row, m, l, acc);
    }
}

template <class K, class... P> hipError_t launch(K kern, size_t x, int threads, size_t lds, hipStream_t st, const P&... p) {
    if (x * threads > 0xffffffffu) return hipErrorInvalidConfiguration;
    if (lds > 65536) {
        const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kern, dim3((unsigned)x), dim3(threads), lds, st, p...);
    return hipGetLastError();
}

// Rows of a block: as many as the longest run of rows that a sequence can have
// fills (a packed batch: its mean). Up to 32 rows go to 16x16 tiles: the other kernel is
// quicker for 32 rows in bf16 at 128 channels (8 sequences of 8 tokens over 8,192, 16 and 4
// heads: 40 us against 45; 64 over 4,096, 32 and 8 heads: 205 and 215) and slower elsewhere (256
// of 5 tokens over 2,048: 414 and 379; 64 of 8 at 64 channels 125 and 120, at 32 103 and 88, in
// fp32 843 and 481).
int block_rows(int T, int N, int G, bool packed) {
    const long rows = packed ? ((long)T + N - 1) / N * G : (long)T * G;
    return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
}
// Workgroups that share the keys: as many as the chip's 256 CUs hold at once of the kernel for
// more rows, so that each is given its share in the same turn. fp32 with 64 rows at 128 channels
// has LDS for one a CU: 8 trees of 12 tokens over 8,192, 16 and 4 heads, 129 us, with two 141; 64
// of 16 over 100 to 4,096, 32 and 8 heads, 462 and 475. Of the kernel for few rows one a CU, also
// where it has registers for two (bf16 at 32 channels: 64 single tokens over 100 to 4,096 49 us,
// with two 43; 8 trees of 8 over 8,192 21 and 23).
template <class T, int D, int R> constexpr int shared_wgs() {
    if constexpr (R <= 32) return 256;
    else return 256 * rows_at_once<T, D, R / 32>();
}
constexpr int most_shared_wgs(int R) { return R <= 32 ? 256 : 512; }   // of any type and head size
// kv heads that the waves of a workgroup take side by side
int heads_together(int Hkv, int waves) {
    int hw = waves;
    while (Hkv % hw) hw /= 2;
    return hw;
}

struct Plan {
    int R;
    long blocks;
    bool shared;
};
// Keys are shared out among workgroups, or every block of rows and head (group) is a
// workgroup's own. bf16, 128 channels, 32 / 8 heads, shared and then not, us. Few rows:
// 400 sequences of 100 to 4,096 tokens 591 and 821, 900 of 100 to 2,048 688 and 795:
// shared as long as the plan can count the blocks. More rows, items of 64 sequences of
// 100 to 8,192 tokens with 32 new ones (512 items) 312 and 391, of 100 sequences (800) 482 and
// 613; from 1,024 items on they fill the chip by themselves, and the parts' sums cost more than
// the evener split gives: 128 sequences of 2,048 tokens with 16 new ones 225 and 219, prompts of
// 16 x 512 tokens (16 / 4 heads) 78 and 51.
Plan make_plan(int T, int N, int Hkv, int G, bool packed) {
    Plan pl;
    pl.R = block_rows(T, N, G, packed);
    pl.blocks = row_blocks_bound(T, N, G, pl.R, packed);
    const long items = pl.blocks * Hkv;
    pl.shared = pl.blocks <= MAX_BLOCKS && items * pl.R < 1 << 24 && (pl.R <= 32 || items < 1024);
    return pl;
}

template <class T, int D, int R> hipError_t attend(const PagedArgs& a, Plan pl) {
    AttnParams p{};
    p.q = a.q; p.Kp = a.Kp; p.Vp = a.Vp; p.ctx = a.ctx; p.tree = a.tree; p.out = a.out; p.lse = a.lse;
    p.pages = make_pages(a);
    p.map = SeqMap{a.cu_seqlens, a.T, a.N};
    p.Hq = a.Hq; p.Hkv = a.Hkv; p.G = a.Hq / a.Hkv; p.words = a.words;
    p.HW = 1;
    if constexpr (R <= 32) p.HW = heads_together(a.Hkv, Few<T, D, R / 16>::NW);
    p.groups = a.Hkv / p.HW;
    p.capacity = std::min((long)a.width * a.page_size, 0x7ffff000L);
    p.scale = a.scale;
    p.blocks = (int)pl.blocks;
    if ((p.capacity / 32 + 1) * pl.blocks > 0x7fffffffL) pl.shared = false;   // units are counted in 31 bits
    const size_t items = (size_t)pl.blocks * p.groups;
    if (pl.shared) {
        p.wgs = shared_wgs<T, D, R>();
        static_assert(shared_wgs<T, D, R>() <= most_shared_wgs(R), "");
        char* ws = static_cast<char*>(a.workspace);
        p.span = reinterpret_cast<int2*>(ws);
        ws += al256(items * 8);
        p.pml = reinterpret_cast<float*>(ws);
        ws += al256((size_t)2 * p.wgs * p.HW * R * 8);
        p.po = reinterpret_cast<float*>(ws);
    }
    const size_t wgs = pl.shared ? p.wgs : items;
    hipError_t e;
    if constexpr (R <= 32) e = launch(paged_few_kernel<T, D, R / 16>, wgs, 64 * Few<T, D, R / 16>::NW, Few<T, D, R / 16>::lds, a.stream, p);
    else e = launch(paged_rows_kernel<T, D, R / 32>, wgs, 256, rows_lds<T, D, R / 32>(), a.stream, p);
    if (e != hipSuccess || !pl.shared) return e;
    const size_t heads = (size_t)pl.blocks * a.Hkv;
    const int rows = a.cu_seqlens ? R : std::min(R, a.T * p.G), room = 1024 / D;   // rows that a block can have
    if (heads * rows <= 1024) return launch(paged_join_kernel<T, D, R, true>, heads * rows, 256, 0, a.stream, p, rows);
    const int J = (rows + room - 1) / room;
    return launch(paged_join_kernel<T, D, R, false>, heads * J, 256, 0, a.stream, p, J);
}

template <class T, int D> hipError_t attend(const PagedArgs& a) {
    const Plan pl = make_plan(a.T, a.N, a.Hkv, a.Hq / a.Hkv, a.cu_seqlens != nullptr);
    return pl.R == 16 ? attend<T, D, 16>(a, pl) : pl.R == 32 ? attend<T, D, 32>(a, pl)
         : pl.R == 64 ? attend<T, D, 64>(a, pl) : attend<T, D, 128>(a, pl);
}

template <class T, int D> hipError_t append(const PagedArgs& a) {
    AppendParams p{};
    p.q = a.q; p.k = a.k; p.v = a.v; p.q_out = a.out; p.Kp = a.Kw; p.Vp = a.Vw;
    p.pos = a.pos; p.ctx = a.ctx; p.freqs = a.freqs;
    p.pages = make_pages(a);
    p.map = SeqMap{a.cu_seqlens, a.T, a.N};
    p.rows = a.cu_seqlens ? a.T : a.N * a.T;
    p.Hq = a.Hq; p.Hkv = a.Hkv; p.rot = a.rot_dim;
    const size_t wgs = std::min(((size_t)p.rows + 3) / 4, (size_t)0xffffff);   // of 256 threads: fewer than 2^32
    return launch(paged_append_kernel<T, D>, wgs, 256, 0, a.stream, p, a.neighbours);
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
    return pl.shared || pl.blocks * Hkv < 1 << 23;
}

size_t paged_attn_workspace_bytes(int T, int N, int Hq, int Hkv, int d, bool packed) {
    const Plan pl = make_plan(T, N, Hkv, Hq / Hkv, packed);
    if (!pl.shared) return 256;
    const size_t slots = (size_t)2 * most_shared_wgs(pl.R) * pl.R * (pl.R <= 32 ? heads_together(Hkv, 8) : 1);
    return al256((size_t)pl.blocks * Hkv * 8) + al256(slots * 8) + slots * d * 4 + 256;
}

hipError_t launch_paged_append(const PagedArgs& a) {
    return KDA_PAGED_DIM(a.d, D, [&] { return a.bf16 ? append<uint16_t, D>(a) : append<float, D>(a); });
}
hipError_t launch_paged_attn(const PagedArgs& a) {
    return KDA_PAGED_DIM(a.d, D, [&] { return a.bf16 ? attend<uint16_t, D>(a) : attend<float, D>(a); });
}

}  // namespace kda
