// Gated linear recurrence for each channel, h_t = a_t h_{t-1} + x_t.
//
// A stretch of tokens acts on the state that enters it as h -> P h + E, with P
// the product of its decays and E its end state from nothing, and two stretches
// compose to another, so that blocks of tokens are taken in parallel: (1) every
// block's P and E, (2) the state that enters each block, one after the other,
// (3) every block again from that state. The gradient has the same form
// backwards: with g the adjoint that enters a token from behind,
//   lam_t = dh_t + g,  dx_t = lam_t,  da_t = lam_t h_{t-1},  g <- a_t lam_t,
// and a block takes g to P g + F. h_{t-1} is formed again from a and x in fp32.
//
// In a block, a thread owns V channels and R consecutive tokens (a slot); slots
// are joined through LDS in the same way.
#include <algorithm>
#include <type_traits>

#include "kda_launch.h"
#include "kda_tiles.h"

namespace kda {

namespace {

constexpr int TILE = 64;    // channels of a workgroup: 128 bytes of a bf16 row
constexpr int NT = 256;     // threads of a workgroup

struct GlrParams {
    const void *gate, *x, *dh;
    const float *h0, *dhT;
    void *h, *dgate, *dx;
    float *hT, *dh0;
    float* sum;             // [block][P, E, F or P, E][C]; E and F become what enters the block
    SeqMap map;
    int C, tiles;
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

// How a workgroup's threads lie over a block of ROWS tokens and TILE channels.
template <int V, int R> struct Lay {
    static constexpr int CL = TILE / V, SLOTS = NT / CL, ROWS = SLOTS * R;
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

// ---------------------------------------------------------------- blocks' P, E and F

template <class TG, class TX, int V, int R, bool GRAD> __global__ void __launch_bounds__(NT) glr_sum_kernel(GlrParams p) {
    using L = Lay<V, R>;
    lds_poison(0);
    __shared__ float sP[L::SLOTS][TILE], sE[L::SLOTS][TILE], sF[GRAD ? L::SLOTS : 1][TILE];
    const int v = blockIdx.x / p.tiles, c0 = blockIdx.x % p.tiles * TILE, tid = threadIdx.x;
    SeqBlock b;
    if (!seq_block(p.map, L::ROWS, v, b)) return;
    const int cl = tid % L::CL * V, slot = tid / L::CL, row = slot * R, c = c0 + cl;
    const bool live = c < p.C;
    const int n = min(b.n - row, R);   // this slot's tokens (or less than none)
    const Rows<TG> ga(p.gate, b.t0, b.n, p.C, row, c, live);
    const Rows<TX> gx(p.x, b.t0, b.n, p.C, row, c, live), gd(p.dh, b.t0, b.n, p.C, row, c, live);
    Raw<TG, V> a[R];
    Raw<TX, V> x[R], d[GRAD ? R : 1];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        a[r].load(ga.rs, ga[r]);
        x[r].load(gx.rs, gx[r]);
        if constexpr (GRAD) d[r].load(gd.rs, gd[r]);
    }
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
#pragma unroll
    for (int i = 0; i < V; ++i) {
        sP[slot][cl + i] = P[i];
        sE[slot][cl + i] = E[i];
        if constexpr (GRAD) sF[slot][cl + i] = F[i];
    }
    __syncthreads();
    if (tid >= (GRAD ? 2 : 1) * TILE || c0 + tid % TILE >= p.C) return;
    const int ch = tid % TILE;
    float* const out = p.sum + (size_t)v * (GRAD ? 3 : 2) * p.C + c0 + ch;
    if (tid < TILE) {
        float pr = 1.f, e = 0.f;
#pragma unroll 8
        for (int s = 0; s < L::SLOTS; ++s) {
            e = fmaf(sP[s][ch], e, sE[s][ch]);
            pr *= sP[s][ch];
        }
        out[0] = pr;
        out[p.C] = e;
    } else {
        float f = 0.f;
#pragma unroll 8
        for (int s = L::SLOTS - 1; s >= 0; --s) f = fmaf(sP[s][ch], f, sF[s][ch]);
        out[2 * p.C] = f;
    }
}

// ---------------------------------------------------------------- what enters each block

// A wave takes 64 channels of one sequence through its blocks, in the gradient
// a second wave backwards. The end state and the first adjoint are results.
template <bool GRAD> __global__ void __launch_bounds__(128) glr_chain_kernel(GlrParams p, int rows) {
    lds_poison(0);
    const int seq = blockIdx.x / p.tiles, c = blockIdx.x % p.tiles * TILE + threadIdx.x % TILE;
    const bool back = threadIdx.x >= TILE;
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
    constexpr int K = GRAD ? 3 : 2, U = 8;
    const size_t step = (size_t)K * p.C;
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
    float* const to = back ? p.dh0 : p.hT;
    if (to) to[at] = h;
}

// ---------------------------------------------------------------- blocks from what enters them

template <class TG, class TX, int V, int R, bool GRAD> __global__ void __launch_bounds__(NT) glr_block_kernel(GlrParams p) {
    using L = Lay<V, R>;
    lds_poison(0);
    __shared__ float sP[L::SLOTS][TILE], sE[L::SLOTS][TILE], sF[GRAD ? L::SLOTS : 1][TILE];
    const int v = blockIdx.x / p.tiles, c0 = blockIdx.x % p.tiles * TILE, tid = threadIdx.x;
    SeqBlock b;
    if (!seq_block(p.map, L::ROWS, v, b)) return;
    const int cl = tid % L::CL * V, slot = tid / L::CL, row = slot * R, c = c0 + cl;
    const bool live = c < p.C;
    const int n = min(b.n - row, R);
    const Rows<TG> ga(p.gate, b.t0, b.n, p.C, row, c, live);
    const Rows<TX> gx(p.x, b.t0, b.n, p.C, row, c, live), gd(p.dh, b.t0, b.n, p.C, row, c, live);
    Raw<TG, V> a[R];
    Raw<TX, V> x[R], d[GRAD ? R : 1];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        a[r].load(ga.rs, ga[r]);
        x[r].load(gx.rs, gx[r]);
        if constexpr (GRAD) d[r].load(gd.rs, gd[r]);
    }
    float carry = 0.f;
    const int ch = tid % TILE;
    if (tid < (GRAD ? 2 : 1) * TILE && c0 + ch < p.C)
        carry = p.sum[((size_t)v * (GRAD ? 3 : 2) + 1 + tid / TILE) * p.C + c0 + ch];
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
#pragma unroll
    for (int i = 0; i < V; ++i) {
        sP[slot][cl + i] = P[i];
        sE[slot][cl + i] = E[i];
        if constexpr (GRAD) sF[slot][cl + i] = F[i];
    }
    __syncthreads();
    if (tid < TILE) {
#pragma unroll 8
        for (int s = 0; s < L::SLOTS; ++s) {
            const float e = sE[s][ch];
            sE[s][ch] = carry;
            carry = fmaf(sP[s][ch], carry, e);
        }
    } else if (GRAD && tid < 2 * TILE) {
#pragma unroll 8
        for (int s = L::SLOTS - 1; s >= 0; --s) {
            const float f = sF[s][ch];
            sF[s][ch] = carry;
            carry = fmaf(sP[s][ch], carry, f);
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i) E[i] = sE[slot][cl + i];
    if constexpr (!GRAD) {
        const Rows<TX> gh(p.h, b.t0, b.n, p.C, row, c, live);
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int i = 0; i < V; ++i) E[i] = fmaf(a[r][i], E[i], x[r][i]);
            Raw<TX, V>::store(gh.rs, gh[r], E);
        }
    } else {
        const Rows<TG> oa(p.dgate, b.t0, b.n, p.C, row, c, live);
        const Rows<TX> ox(p.dx, b.t0, b.n, p.C, row, c, live);
        float before[R][V];
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                before[r][i] = E[i];
                E[i] = fmaf(a[r][i], E[i], x[r][i]);
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) F[i] = sF[slot][cl + i];
#pragma unroll
        for (int r = R - 1; r >= 0; --r) {
            if (r < n) {
                float lam[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    lam[i] = d[r][i] + F[i];
                    F[i] = a[r][i] * lam[i];
                    before[r][i] *= lam[i];
                }
                Raw<TX, V>::store(ox.rs, ox[r], lam);
                Raw<TG, V>::store(oa.rs, oa[r], before[r]);
            }
        }
    }
}

// ---------------------------------------------------------------- one token

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
template <bool WIDE> constexpr int glr_r() { return WIDE ? 4 : 16; }

template <class F> auto with_types(bool bf16, bool gate_bf16, bool wide, F f) {
    using U = uint16_t;
    if (!bf16) return wide ? f(float{}, float{}, std::true_type()) : f(float{}, float{}, std::false_type());
    if (gate_bf16) return wide ? f(U{}, U{}, std::true_type()) : f(U{}, U{}, std::false_type());
    return wide ? f(float{}, U{}, std::true_type()) : f(float{}, U{}, std::false_type());
}

bool wide_rows(int C, bool bf16) { return C % (bf16 ? 8 : 4) == 0; }
int block_rows(int C, bool bf16) {
    if (!wide_rows(C, bf16)) return Lay<1, glr_r<false>()>::ROWS;
    return bf16 ? Lay<8, glr_r<true>()>::ROWS : Lay<4, glr_r<true>()>::ROWS;
}

hipError_t run(const GlrArgs& a, bool grad) {
    GlrParams p{};
    p.gate = a.gate; p.x = a.x; p.dh = a.dh; p.h0 = a.h0; p.dhT = a.dhT;
    p.h = a.h; p.dgate = a.g_gate; p.dx = a.g_x; p.hT = a.hT; p.dh0 = a.g_h0;
    p.sum = static_cast<float*>(a.workspace);
    p.map = SeqMap{a.cu_seqlens, a.T, a.N};
    p.C = a.C;
    p.tiles = (a.C + TILE - 1) / TILE;
    const int rows = block_rows(a.C, a.bf16);
    const unsigned wgs = (unsigned)(seq_blocks_bound(a.T, a.N, rows, a.cu_seqlens != nullptr) * p.tiles);
    return with_types(a.bf16, a.gate_bf16, wide_rows(a.C, a.bf16), [&](auto tg, auto tx, auto wide) {
        using TG = decltype(tg);
        using TX = decltype(tx);
        constexpr int V = glr_v<TX, wide.value>(), R = glr_r<wide.value>();
        if (a.T > 0) {
            if (grad) hipLaunchKernelGGL((glr_sum_kernel<TG, TX, V, R, true>), dim3(wgs), dim3(NT), 0, a.stream, p);
            else hipLaunchKernelGGL((glr_sum_kernel<TG, TX, V, R, false>), dim3(wgs), dim3(NT), 0, a.stream, p);
        }
        const dim3 chains((unsigned)p.tiles * a.N);
        if (grad) hipLaunchKernelGGL((glr_chain_kernel<true>), chains, dim3(2 * TILE), 0, a.stream, p, rows);
        else hipLaunchKernelGGL((glr_chain_kernel<false>), chains, dim3(TILE), 0, a.stream, p, rows);
        if (a.T > 0) {
            if (grad) hipLaunchKernelGGL((glr_block_kernel<TG, TX, V, R, true>), dim3(wgs), dim3(NT), 0, a.stream, p);
            else hipLaunchKernelGGL((glr_block_kernel<TG, TX, V, R, false>), dim3(wgs), dim3(NT), 0, a.stream, p);
        }
        return hipGetLastError();
    });
}

}  // namespace

bool glr_fits(int T, int N, int C, bool packed, bool bf16) {
    const long tiles = (C + TILE - 1) / TILE;
    return (seq_blocks_bound(T, N, block_rows(C, bf16), packed) + N) * tiles * NT <= 0xffffffffL;
}

size_t glr_workspace_bytes(int T, int N, int C, bool packed, bool bf16, bool grad) {
    return (size_t)seq_blocks_bound(T, N, block_rows(C, bf16), packed) * C * (grad ? 12 : 8) + 256;
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
