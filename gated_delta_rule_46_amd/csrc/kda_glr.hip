// Gated linear recurrence for each channel, h_t = a_t h_{t-1} + x_t.
//
// A stretch of tokens acts on the state that enters it as h -> P h + E, with P
// the product of its decays and E its end state from nothing, and two stretches
// compose to another, so that blocks of tokens are taken in parallel.
//
// Forward: one pass. A block's workgroup keeps its values in registers, leaves the
// block's P and E for the blocks behind, takes up those that the blocks before have
// left, and finishes. Gradient: backwards, with g the adjoint that enters a token
// from behind,
//   lam_t = dh_t + g,  dx_t = lam_t,  da_t = lam_t h_{t-1},  g <- a_t lam_t,
// a block takes g to P g + F; one kernel forms every block's P, E and F, another goes
// through every block again from what enters it, which its workgroup forms from the
// other blocks (a long sequence: a kernel of its own, for all blocks). h_{t-1} is formed
// again from a and x in fp32.
//
// In a block, a thread owns V channels and R consecutive tokens (a slot); slots
// are joined through LDS in the same way, one channel a thread. States, products of
// decays and sums are fp32 throughout; results are rounded once.
//
// Bound by memory (2 operations an element). bf16, B=2 C=2048: forward of T=8192 45 us for
// 213 MB at 4.7 TB/s, and 3 to 5 us for the clear before it; gradient of T=4096 20 us (sums,
// 5.1 TB/s) and 32 us (5.2 TB/s): it reads all its inputs twice. (The sums need a and x alone,
// for the states; adjoints could follow each other through one reverse pass as the forward's
// states do, which would save reading dh once, an eighth of the bytes.)
#include <algorithm>
#include <type_traits>

#include "kda_bounds.h"
#include "kda_launch.h"
#include "kda_tiles.h"

namespace kda {

namespace {

constexpr int NT = 256;     // threads of a workgroup
constexpr int WALK = 64;    // gradient: blocks of a sequence whose workgroups form what enters them
constexpr int GROUP = 32;   // forward: blocks that follow each other by P and E, the last one by its state

struct GlrParams {
    const void *gate, *x, *dh;
    const float *h0, *dhT;
    void *h, *dgate, *dx;
    float *hT, *dh0;
    float* sum;             // gradient: [block][P, E, F][C]; E and F become what enters the block
    uint64_t *words, *counter;   // forward: [block][C] what a block has left, and the blocks begun; all ones before
    SeqMap map;
    int C, tiles;
    bool chained;           // sum holds what enters each block
    bool alone;             // no sequence has more than one block, and sum and words are not there
};

// V elements of a row as they lie in memory
template <class T, int V> struct Raw {
    static constexpr int N = V * (int)sizeof(T) / 16;
    u32x4 r[N];
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rs, uint32_t off) {
#pragma unroll
        for (int n = 0; n < N; ++n) r[n] = __builtin_amdgcn_raw_buffer_load_b128(rs, off + 16u * n, 0, 0);
    }
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (sizeof(T) == 2) {
            const uint32_t u = r[i / 8][i / 2 % 4];
            return __uint_as_float(i % 2 ? u & 0xffff0000u : u << 16);
        } else {
            return __uint_as_float(r[i / 4][i % 4]);
        }
    }
    static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t rs, uint32_t off, const float* y) {
        u32x4 o[N];
        T t[V];
#pragma unroll
        for (int i = 0; i < V; ++i) store1(t + i, y[i]);
        __builtin_memcpy(o, t, sizeof(o));
#pragma unroll
        for (int n = 0; n < N; ++n) __builtin_amdgcn_raw_buffer_store_b128(o[n], rs, off + 16u * n, 0, 0);
    }
};
template <> struct Raw<uint16_t, 1> {
    uint16_t r;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rs, uint32_t off) {
        r = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs, off, 0, 0);
    }
    __device__ __forceinline__ float operator[](int) const { return bf16_bits_to_f32(r); }
    static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t rs, uint32_t off, const float* y) {
        uint16_t t;
        store1(&t, y[0]);
        __builtin_amdgcn_raw_buffer_store_b16((short)t, rs, off, 0, 0);
    }
};
template <> struct Raw<float, 1> {
    uint32_t r;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rs, uint32_t off) {
        r = __builtin_amdgcn_raw_buffer_load_b32(rs, off, 0, 0);
    }
    __device__ __forceinline__ float operator[](int) const { return __uint_as_float(r); }
    static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t rs, uint32_t off, const float* y) {
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(y[0]), rs, off, 0, 0);
    }
};

// How a workgroup's threads lie over a block of ROWS tokens and TILE channels (256 bytes of
// a row where rows are read 16 bytes a lane).
template <int V, int R> struct Lay {
    static constexpr int CL = V == 1 ? 64 : 16, TILE = CL * V, SLOTS = NT / CL, ROWS = SLOTS * R;
};

// A block of an array [tokens, C]: rows of a descriptor that ends behind its
// last token; a channel behind C gets an offset behind that end. Loads from
// there are zero and stores go nowhere.
template <class T> struct Rows {
    __amdgpu_buffer_rsrc_t rs;
    uint32_t off, step;
    __device__ __forceinline__ Rows(const void* base, long t0, int n, int C, int row, int c, bool live) {
        const uint32_t bytes = (uint32_t)C * sizeof(T);
        rs = make_rsrc(static_cast<const T*>(base) + (size_t)t0 * C, __builtin_amdgcn_readfirstlane((int)((uint32_t)n * bytes)));
        step = bytes;
        off = live ? (uint32_t)row * bytes + (uint32_t)c * (uint32_t)sizeof(T) : 0xf0000000u;
    }
    __device__ __forceinline__ uint32_t operator[](int r) const { return off + r * step; }
};

// ---------------------------------------------------------------- a block

// A thread's slot of a block: its values, what the slot does to h and g, and the joint of
// the workgroup's slots.
template <class TG, class TX, int V, int R, bool GRAD> struct Block {
    using L = Lay<V, R>;
    static constexpr int TILE = L::TILE, SLOTS = L::SLOTS, K = GRAD ? 3 : 2;
    struct Shared {
        float P[SLOTS][TILE], E[SLOTS][TILE], F[GRAD ? SLOTS : 1][TILE];
    };
    Raw<TG, V> a[R];
    Raw<TX, V> x[R], d[GRAD ? R : 1];
    int cl, slot, c, n;   // first channel in the tile and of all, this slot's tokens (or less than none)
    long t0;
    int rows;
    bool live;

    __device__ __forceinline__ void at(const GlrParams& p, long first, int tokens, int c0) {
        // (said to be the same in every lane: descriptors stay in scalar registers)
        t0 = ((long)__builtin_amdgcn_readfirstlane((int)(first >> 32)) << 32) | (uint32_t)__builtin_amdgcn_readfirstlane((int)first);
        rows = __builtin_amdgcn_readfirstlane(tokens);
        cl = threadIdx.x % L::CL * V;
        slot = threadIdx.x / L::CL;
        c = c0 + cl;
        live = c < p.C;
        n = min(rows - slot * R, R);
    }
    template <class T> __device__ __forceinline__ Rows<T> of(const GlrParams& p, const void* base) const {
        return Rows<T>(base, t0, rows, p.C, slot * R, c, live);
    }
    __device__ __forceinline__ void load(const GlrParams& p) {
        const Rows<TG> ga = of<TG>(p, p.gate);
        const Rows<TX> gx = of<TX>(p, p.x);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            a[r].load(ga.rs, ga[r]);
            x[r].load(gx.rs, gx[r]);
        }
        if constexpr (GRAD) {
            const Rows<TX> gd = of<TX>(p, p.dh);
#pragma unroll
            for (int r = 0; r < R; ++r) d[r].load(gd.rs, gd[r]);
        }
    }
    // the slot's P, E and F
    __device__ __forceinline__ void put(Shared& s) const {
        float P[V], E[V], F[V];
#pragma unroll
        for (int i = 0; i < V; ++i) P[i] = 1.f, E[i] = 0.f, F[i] = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (r < n) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    E[i] = fmaf(a[r][i], E[i], x[r][i]);
                    P[i] *= a[r][i];
                }
            }
        }
        if constexpr (GRAD) {
#pragma unroll
            for (int r = R - 1; r >= 0; --r) {
                if (r < n) {
#pragma unroll
                    for (int i = 0; i < V; ++i) F[i] = a[r][i] * (d[r][i] + F[i]);
                }
            }
        }
        keep(s.P[slot], P);
        keep(s.E[slot], E);
        if constexpr (GRAD) keep(s.F[slot], F);
    }
    __device__ __forceinline__ void keep(float* to, const float* y) const {
        if constexpr (V == 1) to[cl] = y[0];
        else
#pragma unroll
            for (int i = 0; i < V; i += 4) *reinterpret_cast<f32x4*>(to + cl + i) = f32x4{y[i], y[i + 1], y[i + 2], y[i + 3]};
    }
    __device__ __forceinline__ void take(const float* from, float* y) const {
        if constexpr (V == 1) y[0] = from[cl];
        else
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const f32x4 q = *reinterpret_cast<const f32x4*>(from + cl + i);
#pragma unroll
                for (int m = 0; m < 4; ++m) y[i + m] = q[m];
            }
    }
};

// gradient: every block's P, E and F (reads a, x and dh once: 100 MB in 20 us)
template <class TG, class TX, int V, int R> __global__ void __launch_bounds__(NT) glr_sum_kernel(GlrParams p) {
    using B = Block<TG, TX, V, R, true>;
    lds_poison(0);
    __shared__ __align__(16) typename B::Shared s;
    const int v = blockIdx.x / p.tiles, c0 = blockIdx.x % p.tiles * B::TILE, ch = threadIdx.x % B::TILE;
    SeqBlock b;
    if (!seq_block(p.map, B::L::ROWS, v, b)) return;
    B k;
    k.at(p, b.t0, b.n, c0);
    k.load(p);
    k.put(s);
    __syncthreads();
    const int part = threadIdx.x / B::TILE;
    if (part >= 2 || c0 + ch >= p.C) return;
    float* const out = p.sum + (size_t)v * 3 * p.C + c0 + ch;
    if (part == 0) {
        float pr = 1.f, e = 0.f;
#pragma unroll 8
        for (int i = 0; i < B::SLOTS; ++i) {
            e = fmaf(s.P[i][ch], e, s.E[i][ch]);
            pr *= s.P[i][ch];
        }
        out[0] = pr;
        out[p.C] = e;
    } else {
        float f = 0.f;
#pragma unroll 8
        for (int i = B::SLOTS - 1; i >= 0; --i) f = fmaf(s.P[i][ch], f, s.F[i][ch]);
        out[2 * (size_t)p.C] = f;
    }
}

// What a run of `count` blocks, each `step` on in p.sum (backwards where negative), does to h
// (or g): y -> P y + E.
struct Run { float P, E; };
__device__ __forceinline__ Run run_of(const float* P, const float* E, long step, int count) {
    Run r{1.f, 0.f};
    constexpr int U = 8;
    for (int b0 = 0; b0 < count; b0 += U) {
        float pr[U], e[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long o = min(b0 + u, count - 1) * step;
            pr[u] = P[o];
            e[u] = E[o];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (b0 + u < count) {
                r.E = fmaf(pr[u], r.E, e[u]);
                r.P *= pr[u];
            }
        }
    }
    return r;
}

// Gradient of long sequences: what enters each block, in place of its E and F. The first
// wave takes a channel a lane of one sequence through its blocks, the second backwards.
__global__ void __launch_bounds__(128) glr_chain_kernel(GlrParams p, int rows) {
    lds_poison(0);
    const int wide = (p.C + 63) / 64;
    const int seq = blockIdx.x / wide, c = blockIdx.x % wide * 64 + threadIdx.x % 64;
    const bool back = threadIdx.x >= 64;
    if (c >= p.C) return;
    int first, len;
    if (p.map.cu) {
        const int t0 = seq_offset(p.map, seq);
        first = t0 / rows + seq;
        len = max(seq_offset(p.map, seq + 1) - t0, 0);
    } else {
        len = p.map.T;
        first = seq * ((len + rows - 1) / rows);
    }
    const int nb = (len + rows - 1) / rows;
    constexpr int U = 8;
    const size_t step = (size_t)3 * p.C;
    float* const sum = p.sum + first * step + c;
    const size_t at = (size_t)seq * p.C + c;
    const float* const from = back ? p.dhT : p.h0;
    float h = from ? from[at] : 0.f;
    float* const q = sum + (back ? 2 : 1) * (size_t)p.C;
    for (int b0 = 0; b0 < nb; b0 += U) {
        float P[U], E[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int b = min(b0 + u, nb - 1);
            const size_t o = (size_t)(back ? nb - 1 - b : b) * step;
            P[u] = sum[o];
            E[u] = q[o];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int b = b0 + u;
            if (b < nb) {
                q[(size_t)(back ? nb - 1 - b : b) * step] = h;
                h = fmaf(P[u], h, E[u]);
            }
        }
    }
    if (back && p.dh0) p.dh0[at] = h;
}

// a call without tokens: states as they came
__global__ void __launch_bounds__(NT) glr_copy_kernel(const float* from, float* to, size_t n) {
    lds_poison(0);
    const size_t i = (size_t)blockIdx.x * NT + threadIdx.x;
    if (i < n) to[i] = from ? from[i] : 0.f;
}

// gradient: every block from what enters it
template <class TG, class TX, int V, int R> __global__ void __launch_bounds__(NT) glr_grad_kernel(GlrParams p) {
    using B = Block<TG, TX, V, R, true>;
    constexpr int TILE = B::TILE, SLOTS = B::SLOTS;
    lds_poison(0);
    __shared__ __align__(16) typename B::Shared s;
    const int v = blockIdx.x / p.tiles, c0 = blockIdx.x % p.tiles * TILE, ch = threadIdx.x % TILE, part = threadIdx.x / TILE;
    SeqBlock b;
    const bool any = seq_block(p.map, B::L::ROWS, v, b);
    const size_t at = (size_t)b.seq * p.C + c0 + ch;
    const bool mine = part < 2 && c0 + ch < p.C;   // a channel a thread: the first part forwards, the second backwards
    if (!any) {
        if (b.idx == 0 && b.len == 0 && mine && part == 0 && p.dh0) p.dh0[at] = p.dhT ? p.dhT[at] : 0.f;
        return;
    }
    B k;
    k.at(p, b.t0, b.n, c0);
    k.load(p);
    const int nb = (b.len + B::L::ROWS - 1) / B::L::ROWS;
    const long step = 3 * (long)p.C;
    const float* const sum = p.sum + (size_t)v * step + c0 + ch;   // this block's
    float carry = 0.f;
    if (mine && p.chained) {
        carry = sum[(size_t)(1 + part) * p.C];
    } else if (mine) {
        const int count = part ? nb - 1 - b.idx : b.idx;   // blocks on the way from the sequence's end or start
        const float* const first = part ? sum + count * step : sum - count * step;
        const Run r = run_of(first, first + (size_t)(1 + part) * p.C, part ? -step : step, count);
        const float* const from = part ? p.dhT : p.h0;
        carry = fmaf(r.P, from ? from[at] : 0.f, r.E);
    }
    k.put(s);
    __syncthreads();
    if (mine && part == 0) {
#pragma unroll 8
        for (int i = 0; i < SLOTS; ++i) {
            const float e = s.E[i][ch];
            s.E[i][ch] = carry;
            carry = fmaf(s.P[i][ch], carry, e);
        }
    } else if (mine) {
#pragma unroll 8
        for (int i = SLOTS - 1; i >= 0; --i) {
            const float f = s.F[i][ch];
            s.F[i][ch] = carry;
            carry = fmaf(s.P[i][ch], carry, f);
        }
        if (p.dh0 && !p.chained && b.idx == 0) p.dh0[at] = carry;
    }
    __syncthreads();
    float E[V], F[V];
    k.take(s.E[k.slot], E);
    const Rows<TG> oa = k.template of<TG>(p, p.dgate);
    const Rows<TX> ox = k.template of<TX>(p, p.dx);
    float before[R][V];
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            before[r][i] = E[i];
            E[i] = fmaf(k.a[r][i], E[i], k.x[r][i]);
        }
    }
    k.take(s.F[k.slot], F);
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
        if (r < k.n) {
            float lam[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                lam[i] = k.d[r][i] + F[i];
                F[i] = k.a[r][i] * lam[i];
                before[r][i] *= lam[i];
            }
            Raw<TX, V>::store(ox.rs, ox[r], lam);
            Raw<TG, V>::store(oa.rs, oa[r], before[r]);
        }
    }
}

// ---------------------------------------------------------------- forward

constexpr uint64_t NOTHING = ~0ull;   // a word that no block has left yet

__global__ void __launch_bounds__(NT) glr_clear_kernel(uint4* p, size_t n) {
    lds_poison(0);
    const size_t i = (size_t)blockIdx.x * NT + threadIdx.x;
    if (i < n) p[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
}

// P and E (or P = 0 and a state) in one word, so that it is there whole or not at all; no
// NaN is passed on with all bits set
__device__ __forceinline__ void leave(uint64_t* to, float P, float E) {
    const uint32_t e = __float_as_uint(E) == ~0u ? 0x7fc00000u : __float_as_uint(E);
    __hip_atomic_store(to, (uint64_t)e << 32 | __float_as_uint(P), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// What `count` (at most GROUP) words, `step` apart, do to a state, waiting for each to be
// left. All of them belong to workgroups that started earlier and leave them without waiting
// for a later one, so that every wait ends; should one ever not, it gives up after some
// seconds with a NaN.
__device__ __forceinline__ Run take_up(const uint64_t* w, long step, int count) {
    Run r{1.f, 0.f};
    constexpr int U = 8;
    for (int b0 = 0; b0 < count; b0 += U) {
        uint64_t y[U];
        for (int tries = 0;; ++tries) {
            bool all = true;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                y[u] = __hip_atomic_load(w + (long)min(b0 + u, count - 1) * step, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) all &= y[u] != NOTHING;
            if (all || tries == 1 << 22) break;
            __builtin_amdgcn_s_sleep(4);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (b0 + u < count) {
                const float P = __uint_as_float((uint32_t)y[u]), E = __uint_as_float((uint32_t)(y[u] >> 32));
                r.E = fmaf(P, r.E, E);
                r.P *= P;
            }
        }
    }
    return r;
}

// One pass over all blocks. Workgroups take them in the order in which they start (a
// counter), so that a block's predecessors have started before it. A block leaves P and E;
// the first of a sequence, which alone reads h0 (h_T may be h0), and every GROUP-th leave
// the state behind them instead, so that no block looks back over more than GROUP words. Which
// words a block takes up, and in which order, does not depend on when they came. GROUP: one
// sequence of T=131072, C=256 takes 97, 67 and 60 us with states at every 8th, 16th and 32nd
// block. A third workgroup a CU would spill (58 us against 49 at B=2 T=8192 C=2048).
template <class TG, class TX, int V, int R> __global__ void __launch_bounds__(NT) glr_pass_kernel(GlrParams p) {
    using B = Block<TG, TX, V, R, false>;
    constexpr int TILE = B::TILE, SLOTS = B::SLOTS;
    lds_poison(0);
    __shared__ __align__(16) typename B::Shared s;
    __shared__ float s_run[2][TILE], s_in[TILE];
    __shared__ int s_work;
    int work = blockIdx.x;
    if (!p.alone) {
        if (threadIdx.x == 0) s_work = drawn_work(atomicAdd(reinterpret_cast<uint32_t*>(p.counter), 1u), gridDim.x);
        __syncthreads();
        work = __builtin_amdgcn_readfirstlane(s_work);
        if (work < 0) return;   // another call counts here too
    }
    const int v = work / p.tiles, c0 = work % p.tiles * TILE, ch = threadIdx.x % TILE, part = threadIdx.x / TILE;
    SeqBlock b;
    const bool any = seq_block(p.map, B::L::ROWS, v, b);
    const size_t at = (size_t)b.seq * p.C + c0 + ch;
    const bool mine = part < 2 && c0 + ch < p.C;   // a channel a thread, twice
    if (!any) {
        if (b.idx == 0 && b.len == 0 && mine && part == 0 && p.hT) p.hT[at] = p.h0 ? p.h0[at] : 0.f;   // no tokens
        return;
    }
    B k;
    k.at(p, b.t0, b.n, c0);
    k.load(p);
    const bool last = b.idx == (b.len - 1) / B::L::ROWS, head = b.idx == 0;
    const float h0 = head && mine && p.h0 ? p.h0[at] : 0.f;
    k.put(s);
    __syncthreads();
    uint64_t* const word = p.words + (size_t)v * p.C + c0 + ch;   // this block's
    float P = 1.f, E = 0.f;
    if (mine && part == 0) {   // slots' P and E become those of the block up to them
#pragma unroll 8
        for (int i = 0; i < SLOTS; ++i) {
            const float pr = s.P[i][ch], e = s.E[i][ch];
            s.P[i][ch] = P;
            s.E[i][ch] = E;
            E = fmaf(pr, E, e);
            P *= pr;
        }
        if (!last && head) leave(word, 0.f, fmaf(P, h0, E));
        else if (!last && (b.idx + 1) % GROUP) leave(word, P, E);
    }
    if (!head) {   // the words from the last state on, in two halves
        const int first = max(b.idx / GROUP * GROUP - 1, 0), count = b.idx - first, half = (count + 1) / 2;
        if (mine && part == 1) {
            const Run r = take_up(word - (long)(count - half) * p.C, p.C, count - half);
            s_run[0][ch] = r.P;
            s_run[1][ch] = r.E;
        }
        Run r{0.f, 0.f};
        if (mine && part == 0) r = take_up(word - (long)count * p.C, p.C, half);
        __syncthreads();
        if (mine && part == 0) {
            const float h = fmaf(s_run[0][ch], r.E, s_run[1][ch]);
            s_in[ch] = h;
            E = fmaf(P, h, E);
            if (!last && (b.idx + 1) % GROUP == 0) leave(word, 0.f, E);
        }
    } else if (mine && part == 0) {
        s_in[ch] = h0;
        E = fmaf(P, h0, E);
    }
    if (mine && part == 0 && last && p.hT) p.hT[at] = E;
    __syncthreads();
    float h[V], sp[V], se[V];
    k.take(s_in, h);
    k.take(s.P[k.slot], sp);
    k.take(s.E[k.slot], se);
    const Rows<TX> gh = k.template of<TX>(p, p.h);
#pragma unroll
    for (int i = 0; i < V; ++i) h[i] = fmaf(sp[i], h[i], se[i]);
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int i = 0; i < V; ++i) h[i] = fmaf(k.a[r][i], h[i], k.x[r][i]);
        Raw<TX, V>::store(gh.rs, gh[r], h);
    }
}

// Forward of a batch whose sequences and tiles fill the chip: a workgroup takes a tile of
// one sequence through all its blocks, the next one's loads under way, and reads everything
// once. `stream_of` says when it is taken.
template <class TG, class TX, int V, int R> __global__ void __launch_bounds__(NT, 2) glr_stream_kernel(GlrParams p) {
    using B = Block<TG, TX, V, R, false>;
    constexpr int TILE = B::TILE, SLOTS = B::SLOTS, ROWS = B::L::ROWS;
    lds_poison(0);
    __shared__ __align__(16) typename B::Shared s;
    const int seq = blockIdx.x / p.tiles, c0 = blockIdx.x % p.tiles * TILE, ch = threadIdx.x;
    const long first = (long)seq * p.map.T;
    const size_t at = (size_t)seq * p.C + c0 + ch;
    const bool mine = ch < TILE && c0 + ch < p.C;
    float carry = mine && p.h0 ? p.h0[at] : 0.f;
    B k, next;
    next.at(p, first, min(p.map.T, ROWS), c0);
    next.load(p);
    for (int t = 0; t < p.map.T; t += ROWS) {
        k = next;
        if (t + ROWS < p.map.T) {
            next.at(p, first + t + ROWS, min(p.map.T - t - ROWS, ROWS), c0);
            next.load(p);
        }
        k.put(s);
        __syncthreads();
        if (mine) {
#pragma unroll 8
            for (int i = 0; i < SLOTS; ++i) {
                const float e = s.E[i][ch];
                s.E[i][ch] = carry;
                carry = fmaf(s.P[i][ch], carry, e);
            }
        }
        __syncthreads();
        float E[V];
        k.take(s.E[k.slot], E);
        __syncthreads();   // the next block's slots come to the same place
        const Rows<TX> gh = k.template of<TX>(p, p.h);
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int i = 0; i < V; ++i) E[i] = fmaf(k.a[r][i], E[i], k.x[r][i]);
            Raw<TX, V>::store(gh.rs, gh[r], E);
        }
    }
    if (mine && p.hT) p.hT[at] = carry;
}

// ---------------------------------------------------------------- one token

// The state once in and out, with everything else beside it: 256 sequences of 4,096 channels
// bf16 4.0 us for 14.7 MB (a launch's own time is most of it).
template <class TG, class TX, int V> __global__ void __launch_bounds__(NT) glr_decode_kernel(const TG* __restrict__ gate, const TX* __restrict__ x, float* __restrict__ h, TX* __restrict__ o, size_t n) {
    lds_poison(0);
    const size_t at = ((size_t)blockIdx.x * NT + threadIdx.x) * V;
    if (at >= n) return;
    float y[V];
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] = fmaf(from_el(gate[at + i]), h[at + i], from_el(x[at + i]));
#pragma unroll
    for (int i = 0; i < V; ++i) {
        h[at + i] = y[i];
        store1(o + at + i, y[i]);
    }
}

// Channels and tokens of a thread: 16 bytes of the input type where every row
// starts at a multiple of them, else one channel.
template <class TX, bool WIDE> constexpr int glr_v() { return WIDE ? 16 / (int)sizeof(TX) : 1; }
template <bool WIDE> constexpr int glr_r() { return WIDE ? 8 : 16; }
// The forward's single pass takes more: fewer blocks look back, with registers for two
// workgroups a CU. B=2 T=8192 C=2048 bf16, 4, 8, 12 and 16 tokens: 69, 50, 48 and 52 us; B=1
// T=4096 C=2048 fp32, 8, 12 and 16: 30, 26 and 24 us; B=1 T=4096 C=2049 bf16, 16, 32, 48 and 64:
// 38, 29, 24 and 23.
template <int V> constexpr int pass_r() { return V == 8 ? 12 : V == 4 ? 16 : 64; }
constexpr int pass_rows(bool wide, bool bf16) {
    return !wide ? Lay<1, pass_r<1>()>::ROWS : bf16 ? Lay<8, pass_r<8>()>::ROWS : Lay<4, pass_r<4>()>::ROWS;
}
constexpr int grad_rows(bool wide) { return wide ? 128 : 64; }
// The streaming forward holds two blocks. With fp32 decays beside bf16 x eight tokens of each
// spill (B=16 T=4096 C=2048, 4, 6 and 8 tokens: 195, 199 and 289 us).
template <class TG, class TX, bool WIDE> constexpr int stream_r() { return WIDE && sizeof(TG) > sizeof(TX) ? 4 : glr_r<WIDE>(); }

// Whether the forward streams: from 256 pairs of a sequence and a tile on, one a CU, and in fp32
// up to 2^25 values of x. The streaming kernel's us against the single pass's:
//   bf16 (T, 16 of C=2048)      512: 17, 27    1,024: 40, 47    2,048: 81, 85     4,096: 158, 156
//   fp32 decays beside bf16     512: 25, 35    1,024: 47, 57    2,048: 99, 107    4,096: 194, 198
//   fp32                        512: 36, 46    1,024: 80, 84    2,048: 166, 152   4,096: 320, 287
// (fp32, 32 of T=2048 C=1024 and 64 of T=2048 C=509: 159, 152 and 229, 199.) With 128 pairs it is
// slower (bf16, 8 of T=4096 C=2048: 99, 86).
bool stream_of(const GlrArgs& a, int tiles) {
    return !a.cu_seqlens && (long)a.N * tiles >= 256 && (a.bf16 || (long)a.N * a.T * a.C <= 1L << 25);
}

template <class F> auto with_types(bool bf16, bool gate_bf16, bool wide, F f) {
    using U = uint16_t;
    if (!bf16) return wide ? f(float{}, float{}, std::true_type()) : f(float{}, float{}, std::false_type());
    if (gate_bf16) return wide ? f(U{}, U{}, std::true_type()) : f(U{}, U{}, std::false_type());
    return wide ? f(float{}, U{}, std::true_type()) : f(float{}, U{}, std::false_type());
}

bool wide_rows(int C, bool bf16) { return C % (bf16 ? 8 : 4) == 0; }
static_assert(Lay<8, glr_r<true>()>::ROWS == grad_rows(true) && Lay<4, glr_r<true>()>::ROWS == grad_rows(true) &&
              Lay<1, glr_r<false>()>::ROWS == grad_rows(false), "");

hipError_t run(const GlrArgs& a, bool grad) {
    GlrParams p{};
    p.gate = a.gate; p.x = a.x; p.dh = a.dh; p.h0 = a.h0; p.dhT = a.dhT;
    p.h = a.h; p.dgate = a.g_gate; p.dx = a.g_x; p.hT = a.hT; p.dh0 = a.g_h0;
    p.sum = static_cast<float*>(a.workspace);
    p.map = SeqMap{a.cu_seqlens, a.T, a.N};
    p.C = a.C;
    return with_types(a.bf16, a.gate_bf16, wide_rows(a.C, a.bf16), [&](auto tg, auto tx, auto wide) {
        using TG = decltype(tg);
        using TX = decltype(tx);
        constexpr int V = glr_v<TX, wide.value>(), R = glr_r<wide.value>();
        using L = Lay<V, R>;
        p.tiles = (a.C + L::TILE - 1) / L::TILE;
        const bool packed = a.cu_seqlens != nullptr;
        const int rows = grad ? L::ROWS : pass_rows(wide.value, a.bf16);
        const size_t blocks = seq_blocks_bound(a.T, a.N, rows, packed);
        const dim3 wgs((unsigned)(blocks * p.tiles)), nt(NT);
        const int most = (a.T + rows - 1) / rows;   // blocks that one sequence can have
        if (most == 0) {
            const size_t n = (size_t)a.N * a.C;
            hipLaunchKernelGGL(glr_copy_kernel, dim3((unsigned)((n + NT - 1) / NT)), nt, 0, a.stream, grad ? a.dhT : a.h0,
                               grad ? a.g_h0 : a.hT, n);
            return hipGetLastError();
        }
        p.alone = most == 1;
        p.chained = grad && most > WALK;
        if (grad) {
            if (!p.alone) hipLaunchKernelGGL((glr_sum_kernel<TG, TX, V, R>), wgs, nt, 0, a.stream, p);
            if (p.chained) hipLaunchKernelGGL(glr_chain_kernel, dim3((unsigned)((a.C + 63) / 64) * a.N), dim3(128), 0, a.stream, p, rows);
            hipLaunchKernelGGL((glr_grad_kernel<TG, TX, V, R>), wgs, nt, 0, a.stream, p);
            return hipGetLastError();
        }
        if (!p.alone && stream_of(a, p.tiles)) {
            hipLaunchKernelGGL((glr_stream_kernel<TG, TX, V, stream_r<TG, TX, wide.value>()>), dim3(a.N * p.tiles), nt, 0, a.stream, p);
            return hipGetLastError();
        }
        if (!p.alone) {
            p.words = static_cast<uint64_t*>(a.workspace);
            p.counter = p.words + blocks * a.C;
            const size_t n = (blocks * a.C + 2) / 2 + 1;   // 16 bytes each, the counter among them
            hipLaunchKernelGGL(glr_clear_kernel, dim3((unsigned)((n + NT - 1) / NT)), nt, 0, a.stream, static_cast<uint4*>(a.workspace), n);
        }
        hipLaunchKernelGGL((glr_pass_kernel<TG, TX, V, pass_r<V>()>), wgs, nt, 0, a.stream, p);
        return hipGetLastError();
    });
}

}  // namespace

bool glr_fits(int T, int N, int C, bool packed, bool bf16) {
    const long tiles = (C + 63) / 64;
    return (seq_blocks_bound(T, N, grad_rows(wide_rows(C, bf16)), packed) + N) * tiles * NT <= 0xffffffffL;
}

size_t glr_workspace_bytes(int T, int N, int C, bool packed, bool bf16, bool grad) {
    const bool wide = wide_rows(C, bf16);
    return (size_t)seq_blocks_bound(T, N, grad ? grad_rows(wide) : pass_rows(wide, bf16), packed) * C * (grad ? 12 : 8) + 256;
}

hipError_t launch_glr_fwd(const GlrArgs& a) { return run(a, false); }
hipError_t launch_glr_bwd(const GlrArgs& a) { return run(a, true); }

hipError_t launch_glr_decode(const GlrDecodeArgs& a) {
    const size_t n = (size_t)a.N * a.C;
    const bool al = ((uintptr_t)a.gate | (uintptr_t)a.x | (uintptr_t)a.h | (uintptr_t)a.o) % 16 == 0;
    return with_types(a.bf16, a.gate_bf16, al && n % 8 == 0, [&](auto tg, auto tx, auto wide) {
        using TG = decltype(tg);
        using TX = decltype(tx);
        constexpr int V = wide.value ? 8 : 1;
        hipLaunchKernelGGL((glr_decode_kernel<TG, TX, V>), dim3((unsigned)((n / V + NT - 1) / NT)), dim3(NT), 0, a.stream,
                           (const TG*)a.gate, (const TX*)a.x, a.h, (TX*)a.o, n);
        return hipGetLastError();
    });
}

}  // namespace kda
