// Softmax attention over a sliding window with sinks: row i of a sequence sees
// the keys j <= i with i - j < window, and the first `sinks` keys always.
//
//   s_ij = scale q_i . k_j,  p_ij = exp(s_ij - lse_i),  o_i = sum_j p_ij v_j
//
// Every product runs on 32x32 MFMA tiles, 16 deep (bf16; fp32: eight 32x32x2
// steps): lane l = 32 h + n holds row (column) n of an operand at 8 of the 16
// contracted places, and column n of the result at rows 8 (r / 4) + 4 h + r % 4.
// Scores are formed transposed (keys down, queries across), so a lane owns one
// query: its maximum and sum run over the lane's registers and one swap with
// the other half, and the exponentials are the next product's operand as they
// stand, with no pass through LDS (the contraction takes the keys in the order
// in which the registers hold them).
//
// Scores, statistics and sums are fp32. bf16 inputs: p and, in the gradient, p (dP -
// delta) enter the second products rounded to bf16, which takes half the instructions of
// two bf16 numbers and makes about as much error as the rounding of the results: o is off by
// 2.21e-3 of its rms where its own rounding makes 1.63e-3 (T = 8192, window 1024), the
// gradients by 2.34e-3 to 2.36e-3 against 1.66e-3 (T = 4096, window 512).
#include <algorithm>
#include <type_traits>

#include "kda_launch.h"
#include "kda_tiles.h"

typedef float f32x16 __attribute__((ext_vector_type(16)));

namespace kda {

namespace {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

struct SwaParams {
    const void *q, *k, *v, *o, *dO;
    const float* lse;
    void *out, *dq, *dk, *dv;
    float *lse_out, *delta;
    float* part;            // gradients of key blocks in parts: [slot][dv, dk][KB][D]
    SeqMap map;
    int Hq, Hkv, G;         // G = Hq / Hkv
    int HW;                 // heads of a group that a workgroup takes together
    int window, sinks;
    float scale;
    int blocks;             // blocks of rows over all sequences
    int sink_blocks, sink_rows, sink_parts;   // gradient: key blocks with sinks, rows a part of theirs, parts over all sequences
    int head_parts;                        // gradient: parts of a group's query heads
};

__device__ __forceinline__ f32x16 mma32(const bf16x8& a, const bf16x8& b, const f32x16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma32(const f32x8& a, const f32x8& b, f32x16 c) {
#pragma unroll
    for (int m = 0; m < 8; ++m) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[m], b[m], c, 0, 0, 0);
    return c;
}
__device__ __forceinline__ f32x16 zero16() {
    f32x16 z;
#pragma unroll
    for (int r = 0; r < 16; ++r) z[r] = 0.f;
    return z;
}

// rows r0 + n, columns k0 + 8 h + (0..7)
template <class T>
__device__ __forceinline__ typename Frag<T>::V nat32(const T* t, int st, int r0, int k0, int n, int h) {
    return frag_nat(t, st, r0 + n, k0, h);
}
// column c0 + n, rows r0 + 4 h + (0..3) and r0 + 8 + 4 h + (0..3)
__device__ __forceinline__ bf16x8 tr32(const uint16_t* t, int st, int r0, int c0, int lane) {
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const int i = lane & 15, b = (lane >> 4) & 1, h = lane >> 5;
    const uint16_t* p = t + (r0 + 4 * h + (i >> 2)) * st + c0 + 16 * b + 4 * (i & 3);
    const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
    const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 8 * st));
    const auto u = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8, u);
}
__device__ __forceinline__ f32x8 tr32(const float* t, int st, int r0, int c0, int lane) {
    const float* p = t + (r0 + 4 * (lane >> 5)) * st + c0 + (lane & 31);
    f32x8 r;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        r[m] = p[m * st];
        r[4 + m] = p[(8 + m) * st];
    }
    return r;
}
// half b of a result tile's rows as an operand (rows contracted)
template <class T> __device__ __forceinline__ typename Frag<T>::V rows16(const f32x16& x, int b) {
    f32x8 y;
#pragma unroll
    for (int m = 0; m < 8; ++m) y[m] = x[8 * b + m];
    return narrow<T>(y);
}
__device__ __forceinline__ int result_row(int r, int h) { return 8 * (r >> 2) + 4 * h + (r & 3); }

// A lane's values of a result tile, times f, to 32 consecutive columns of a row:
// bf16 halves of 8 columns are swapped with the other half of the wave first, so
// that they go out 16 bytes a lane instead of 8.
template <class T> __device__ __forceinline__ void store_tile(T* row, const f32x16& y, float f, int h) {
#pragma unroll
    for (int r = 0; r < 4; r += 2) {
        const f32x4 a = f32x4{y[4 * r], y[4 * r + 1], y[4 * r + 2], y[4 * r + 3]} * f;
        const f32x4 b = f32x4{y[4 * r + 4], y[4 * r + 5], y[4 * r + 6], y[4 * r + 7]} * f;
        if constexpr (sizeof(T) == 2) {
            u32x2 u, v;
            store4(reinterpret_cast<T*>(&u), a);
            store4(reinterpret_cast<T*>(&v), b);
            const auto s0 = __builtin_amdgcn_permlane32_swap(u[0], v[0], false, false);
            const auto s1 = __builtin_amdgcn_permlane32_swap(u[1], v[1], false, false);
            *reinterpret_cast<uint4*>(row + 8 * (r + h)) = make_uint4(s0[0], s1[0], s0[1], s1[1]);
        } else {
            store4(row + 8 * r + 4 * h, a);
            store4(row + 8 * r + 8 + 4 * h, b);
        }
    }
}

// 8 consecutive elements of a row in global memory, or zeros
template <class T> __device__ __forceinline__ typename Frag<T>::V load8(const T* p, bool in) {
    constexpr int N = sizeof(T) / 2;
    uint4 u[N];
#pragma unroll
    for (int m = 0; m < N; ++m) u[m] = in ? reinterpret_cast<const uint4*>(p)[m] : make_uint4(0u, 0u, 0u, 0u);
    typename Frag<T>::V r;
    __builtin_memcpy(&r, u, sizeof(r));
    return r;
}

__device__ __forceinline__ float swap_max(float v) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float swap_sum(float v) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// largest of 16 values (IEEE maximum: takes a product's result as it is, where
// fmaxf would first quiet every operand with an instruction of its own)
__device__ __forceinline__ float tree_max(const f32x16& x) {
    float m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m[i] = __builtin_elementwise_maximum(__builtin_elementwise_maximum(x[4 * i], x[4 * i + 1]),
                                             __builtin_elementwise_maximum(x[4 * i + 2], x[4 * i + 3]));
    return __builtin_elementwise_maximum(__builtin_elementwise_maximum(m[0], m[1]), __builtin_elementwise_maximum(m[2], m[3]));
}

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }   // 1 ulp, no range fix-up

// keys (rows) per tile that a workgroup stages
template <class T> constexpr int swa_tile() { return sizeof(T) == 2 ? 64 : 32; }

// Whether rows [i0, i1] see none of the keys [j0, j1], or all of them.
struct Seen { bool none, all; };
__device__ __forceinline__ Seen seen(int i0, int i1, int j0, int j1, int window, int sinks) {
    return Seen{j0 > i1 || (i0 - j1 >= window && j0 >= sinks), j1 <= i0 && (i1 - j0 < window || j1 < sinks)};
}
__device__ __forceinline__ bool sees(int i, int j, int window, int sinks) {
    return j <= i && (i - j < window || j < sinks);
}
// The same for one lane and many keys at constant offsets from `j`.
struct Mask {
    int last, first, sink;   // offsets seen: first < c <= last, or c < sink and c <= last
    __device__ __forceinline__ Mask(int i, int j, int window, int sinks) : last(i - j), first(i - j - window), sink(sinks - j) {}
    __device__ __forceinline__ bool operator()(int c) const { return c <= last && (c > first || c < sink); }
};

// The key tiles of rows [q0, q1]: first those with sinks, then the window's.
struct KeyTiles {
    int sink, first, count;
    __device__ __forceinline__ KeyTiles(int q0, int q1, int tile, int window, int sinks) {
        first = max(q0 - window + 1, 0) / tile;
        sink = min((sinks + tile - 1) / tile, first);
        count = sink + q1 / tile - first + 1;
    }
    __device__ __forceinline__ int operator[](int it) const { return it < sink ? it : first + it - sink; }
};

// A workgroup of NW waves takes HW heads of one group (the largest power of two
// that divides both) for 32 NW / HW rows: heads side by side read the same key
// tiles, and the fewer rows they have, the fewer tiles lie across a mask's edge.
// Forward and gradient of 4,096 rows, 16 and 4 heads, d = 128: 0.168 ms with a window of
// 128, 0.173 with a head a workgroup; 0.205 against 0.206 with one of 512.
__host__ __device__ inline int heads_together(int G, int NW) {
    int hw = NW;
    while (G % hw) hw /= 2;
    return hw;
}
// workgroup number -> (block of rows, first head): the heads of one block next
// to each other on one XCD, which keeps the block's keys in its L2; late blocks,
// which see more keys, first
__device__ __forceinline__ void work_item(const SwaParams& p, int& blk, int& head) {
    const int heads = p.Hq / p.HW, e = xcd_remap(blockIdx.x, p.blocks * heads);
    blk = p.blocks - 1 - e / heads;
    head = e % heads * p.HW;
}

// ---------------------------------------------------------------- forward

// NW waves of 32 queries each share the key tiles, staged twice over in LDS
// (one barrier a tile). B = 2, T = 8192, 16 and 4 heads, d = 128, window 1024, 4 sinks,
// bf16: 0.18 to 0.19 ms, 670 to 716 TFLOP/s of what the window holds (half of a large library
// product's rate); bound by the exponentials and the matrix products of two waves a SIMD, which
// overlap only across waves (matrix units busy for 31% of the time).
// KS > 1, for few rows: KS waves take the same 32 queries and every KS-th key tile
// each, and join what they have at the end.
template <class T, int D, int NW, int KS> __global__ void __launch_bounds__(64 * NW) swa_fwd_kernel(SwaParams p) {
    constexpr int KT = swa_tile<T>(), KB = KS * KT, NX = KT / 32, NT = 64 * NW, ST = tile_stride<T>(D), KD = D / 16, MD = D / 32;
    using V8 = typename Frag<T>::V;
    extern __shared__ __align__(16) unsigned char smem[];
    lds_poison((uint32_t)(sizeof(T) * 4 * KB * ST));
    T* const tiles = reinterpret_cast<T*>(smem);   // [2][k, v][KB][ST]

    const int tid = threadIdx.x, lane = tid % WAVE, w = tid / WAVE, n = lane & 31, h2 = lane >> 5;
    int blk, h;
    work_item(p, blk, h);
    const int rows = 32 * (NW / KS) / p.HW, wr = w / KS, wk = w % KS;
    SeqBlock b;
    if (!seq_block(p.map, rows, blk, b)) return;
    const int q0 = b.idx * rows, len = b.len;
    const long ts = b.t0 - q0;
    const int hk = h / p.G;
    h += wr % p.HW;
    const int i0 = q0 + wr / p.HW * 32, row = i0 + n;
    const bool live = row < len;
    // a negative scale goes into q, exactly, so that maxima scale as they stand
    const float c = fabsf(p.scale) * LOG2E;

    V8 qf[KD];
    {
        const T* src = static_cast<const T*>(p.q) + ((size_t)(ts + (live ? row : 0)) * p.Hq + h) * D + 8 * h2;
#pragma unroll
        for (int ks = 0; ks < KD; ++ks) {
            qf[ks] = load8<T>(src + 16 * ks, live);
            if (p.scale < 0.f) qf[ks] = -qf[ks];
        }
    }
    const T* K = static_cast<const T*>(p.k) + ((size_t)ts * p.Hkv + hk) * D;
    const T* V = static_cast<const T*>(p.v) + ((size_t)ts * p.Hkv + hk) * D;
    const size_t rs = (size_t)p.Hkv * D;
    const KeyTiles kt(q0, min(q0 + rows, len) - 1, KB, p.window, p.sinks);

    Stage<T, D, KB, NT> sk, sv;
    auto fetch = [&](int it) {
        const int j0 = kt[it] * KB;
        sk.load(K + (size_t)j0 * rs, rs, len - j0, tid);
        sv.load(V + (size_t)j0 * rs, rs, len - j0, tid);
    };
    auto put = [&](int it) {
        T* t = tiles + (it & 1) * 2 * KB * ST;
        sk.store(t, tid);
        sv.store(t + KB * ST, tid);
    };
    f32x16 O[MD];
#pragma unroll
    for (int m = 0; m < MD; ++m) O[m] = zero16();
    float top = -INFINITY, sum = 0.f;   // sum: this lane's half of the keys

    auto tile = [&](const T* tk, const T* tv, int j0, auto masked) {
        f32x16 s[NX];
        V8 kf[NX][KD], vf[MD];
#pragma unroll
        for (int ks = 0; ks < KD; ++ks)
#pragma unroll
            for (int x = 0; x < NX; ++x) kf[x][ks] = nat32<T>(tk, ST, 32 * x, 16 * ks, n, h2);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int x = 0; x < NX; ++x) s[x] = zero16();
        f32x16 odd = zero16();   // one tile of keys: two chains of products, added
#pragma unroll
        for (int ks = 0; ks < KD; ++ks)
#pragma unroll
            for (int x = 0; x < NX; ++x) {
                if (NX == 1 && ks % 2) odd = mma32(kf[x][ks], qf[ks], odd);
                else s[x] = mma32(kf[x][ks], qf[ks], s[x]);
            }
        if constexpr (NX == 1) s[0] += odd;
#pragma unroll
        for (int m = 0; m < MD; ++m) vf[m] = tr32(tv, ST, 0, 32 * m, lane);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (masked.value) {
            const Mask mask(row, j0 + 4 * h2, p.window, p.sinks);
#pragma unroll
            for (int x = 0; x < NX; ++x)
#pragma unroll
                for (int r = 0; r < 16; ++r) s[x][r] = mask(32 * x + result_row(r, 0)) ? s[x][r] * c : -INFINITY;
        }
        const float f = masked.value ? 1.f : c;   // what is left to scale
        float mt = tree_max(s[0]);
#pragma unroll
        for (int x = 1; x < NX; ++x) mt = __builtin_elementwise_maximum(mt, tree_max(s[x]));
        mt = swap_max(mt * f);
        // The subtracted maximum may lag behind by 2^8: sums stay far inside
        // fp32, and most tiles leave o as it is.
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
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < NX; ++x)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                s[x][r] = fast_exp2(fmaf(s[x][r], f, -base));
                part[r & 3] += s[x][r];
            }
        sum += (part[0] + part[1]) + (part[2] + part[3]);
#pragma unroll
        for (int kb = 0; kb < KT / 16; ++kb) {
            V8 next[MD];
            if (kb + 1 < KT / 16) {
#pragma unroll
                for (int m = 0; m < MD; ++m) next[m] = tr32(tv, ST, 16 * (kb + 1), 32 * m, lane);
            }
            const V8 pf = rows16<T>(s[kb / 2], kb % 2);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int m = 0; m < MD; ++m) O[m] = mma32(vf[m], pf, O[m]);
            if (kb + 1 < KT / 16) {
#pragma unroll
                for (int m = 0; m < MD; ++m) vf[m] = next[m];
            }
        }
    };

    fetch(0);
    put(0);
    __syncthreads();
    for (int it = 0; it < kt.count; ++it) {
        if (it + 1 < kt.count) fetch(it + 1);
        const T* tk = tiles + ((it & 1) * 2 * KB + wk * KT) * ST;
        const T* tv = tk + KB * ST;
        const int j0 = kt[it] * KB + wk * KT;
        const Seen se = seen(i0, i0 + 31, j0, j0 + KT - 1, p.window, p.sinks);
        if (!se.none && i0 < len) {
            if (se.all) tile(tk, tv, j0, std::false_type()); else tile(tk, tv, j0, std::true_type());
        }
        if (it + 1 < kt.count) {
            put(it + 1);
            __syncthreads();
        }
    }
    sum = swap_sum(sum);
    if constexpr (KS > 1) {   // in the tiles' place: [wave][value][lane]
        static_assert((16 * MD + 2) * 4 * 64 * NW <= sizeof(T) * 4 * KB * ST, "room for the join");
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
        if (wk) return;
#pragma unroll
        for (int y = 1; y < KS; ++y) {
            const float* other = join + (size_t)y * (16 * MD + 2) * 64;
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
    // An Inf or NaN in v at a key that a tile holds but a row does not see has
    // entered that row as 0 * v. Rows that are not finite are formed again, one
    // key at a time, from the keys that they see.
    float probe = 0.f;
#pragma unroll
    for (int m = 0; m < MD; ++m)
#pragma unroll
        for (int r = 0; r < 16; ++r) probe += O[m][r] * 0.f;
    if (__any(live && probe != 0.f)) {
#pragma unroll
        for (int m = 0; m < MD; ++m) O[m] = zero16();
        const T* Q = static_cast<const T*>(p.q) + ((size_t)(ts + (live ? row : 0)) * p.Hq + h) * D;
        for (int j = 0; j <= min(i0 + 31, len - 1); ++j) {
            const bool in = live && sees(row, j, p.window, p.sinks);
            if (!__any(in)) continue;
            float dot = 0.f;
            for (int x = 0; x < D; x += 8) {
                const f32x8 y = widen(load8<T>(Q + x, true)) * widen(load8<T>(K + (size_t)j * rs + x, true));
                dot += ((y[0] + y[1]) + (y[2] + y[3])) + ((y[4] + y[5]) + (y[6] + y[7]));
            }
            const float e = fast_exp2(dot * (p.scale * LOG2E) - top);
            if (!in) continue;
#pragma unroll
            for (int m = 0; m < MD; ++m)
#pragma unroll
                for (int r = 0; r < 16; ++r) O[m][r] += e * from_el(V[(size_t)j * rs + 32 * m + result_row(r, h2)]);
        }
    }
    const float inv = 1.f / sum;
    if (live) {
        T* out = static_cast<T*>(p.out) + ((size_t)(ts + row) * p.Hq + h) * D;
#pragma unroll
        for (int m = 0; m < MD; ++m) store_tile<T>(out + 32 * m, O[m], inv, h2);
        if (p.lse_out && h2 == 0) p.lse_out[(size_t)(ts + row) * p.Hq + h] = (top + log2f(sum)) * LN2;
    }
}

// ---------------------------------------------------------------- gradient with respect to q

// As the forward, with dP^T = V dO^T and dS = P (dP - delta), delta_i = dO_i . o_i
// (formed here and kept for the other gradients): dq^T = K^T dS^T; KS as there. With o in
// bf16 that product takes o's rounding into every dS, which where a row attends to few
// keys is as large as dP itself: dq and dk were off by up to 2.3 times their own
// rounding, with scores of deviation 4 also in windows of 1,024. bf16 rows therefore
// walk their keys once more, for delta_i = sum_j p_ij dP_ij in fp32: off by 1.44 at most. 4,096
// rows, 16 and 4 heads, d = 128, window 512, bf16: 66 us, 48 without; the whole gradient of
// windows of 32, 128 and 1,024 71, 141 and 1,416 us against 72, 138 and 1,174.
template <class T, int D, int NW, int KS> __global__ void __launch_bounds__(64 * NW) swa_dq_kernel(SwaParams p) {
    constexpr bool SUMMED = sizeof(T) == 2;
    constexpr int KT = swa_tile<T>(), KB = KS * KT, NT = 64 * NW, ST = tile_stride<T>(D), KD = D / 16, MD = D / 32;
    using V8 = typename Frag<T>::V;
    extern __shared__ __align__(16) unsigned char smem[];
    lds_poison((uint32_t)(sizeof(T) * 4 * KB * ST));
    T* const tiles = reinterpret_cast<T*>(smem);

    const int tid = threadIdx.x, lane = tid % WAVE, w = tid / WAVE, n = lane & 31, h2 = lane >> 5;
    int blk, h;
    work_item(p, blk, h);
    const int rows = 32 * (NW / KS) / p.HW, wr = w / KS, wk = w % KS;
    SeqBlock b;
    if (!seq_block(p.map, rows, blk, b)) return;
    const int q0 = b.idx * rows, len = b.len;
    const long ts = b.t0 - q0;
    const int hk = h / p.G;
    h += wr % p.HW;
    const int i0 = q0 + wr / p.HW * 32, row = i0 + n;
    const bool live = row < len;
    const float c = p.scale * LOG2E;

    V8 qf[KD], gf[KD];
    float delta = 0.f, lse2 = 0.f;
    const size_t r0 = (size_t)(ts + (live ? row : 0)) * p.Hq + h;
    {
        const T* sq = static_cast<const T*>(p.q) + r0 * D + 8 * h2;
        const T* sg = static_cast<const T*>(p.dO) + r0 * D + 8 * h2;
        const T* so = static_cast<const T*>(p.o) + r0 * D + 8 * h2;
#pragma unroll
        for (int ks = 0; ks < KD; ++ks) {
            qf[ks] = load8<T>(sq + 16 * ks, live);
            gf[ks] = load8<T>(sg + 16 * ks, live);
            if constexpr (!SUMMED) {
                const f32x8 x = widen(gf[ks]) * widen(load8<T>(so + 16 * ks, live));
                delta += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
            }
        }
        if (live) lse2 = p.lse[r0] * LOG2E;
    }
    const T* K = static_cast<const T*>(p.k) + ((size_t)ts * p.Hkv + hk) * D;
    const T* V = static_cast<const T*>(p.v) + ((size_t)ts * p.Hkv + hk) * D;
    const size_t rs = (size_t)p.Hkv * D;
    const KeyTiles kt(q0, min(q0 + rows, len) - 1, KB, p.window, p.sinks);

    Stage<T, D, KB, NT> sk, sv;
    auto fetch = [&](int it) {
        const int j0 = kt[it] * KB;
        sk.load(K + (size_t)j0 * rs, rs, len - j0, tid);
        sv.load(V + (size_t)j0 * rs, rs, len - j0, tid);
    };
    auto put = [&](int it) {
        T* t = tiles + (it & 1) * 2 * KB * ST;
        sk.store(t, tid);
        sv.store(t + KB * ST, tid);
    };
    // delta of a tile's keys
    auto sum_tile = [&](const T* tk, const T* tv, int x, int j0, auto masked) {
        f32x16 s = zero16(), d = zero16();
#pragma unroll
        for (int ks = 0; ks < KD; ++ks) {
            s = mma32(nat32<T>(tk, ST, 32 * x, 16 * ks, n, h2), qf[ks], s);
            d = mma32(nat32<T>(tv, ST, 32 * x, 16 * ks, n, h2), gf[ks], d);
        }
        const Mask mask(row, j0 + 4 * h2, p.window, p.sinks);
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const float e = fast_exp2(fmaf(s[r], c, -lse2)) * d[r];
            part[r & 3] += !masked.value || mask(result_row(r, 0)) ? e : 0.f;
        }
        delta += (part[0] + part[1]) + (part[2] + part[3]);
    };
    if constexpr (SUMMED) {
        fetch(0);
        put(0);
        __syncthreads();
        for (int it = 0; it < kt.count; ++it) {
            if (it + 1 < kt.count) fetch(it + 1);
            const T* tk = tiles + ((it & 1) * 2 * KB + wk * KT) * ST;
            const T* tv = tk + KB * ST;
            if (i0 < len) {
#pragma unroll
                for (int x = 0; x < KT / 32; ++x) {
                    const int j0 = kt[it] * KB + wk * KT + 32 * x;
                    const Seen se = seen(i0, i0 + 31, j0, j0 + 31, p.window, p.sinks);
                    if (se.none) continue;
                    if (se.all) sum_tile(tk, tv, x, j0, std::false_type()); else sum_tile(tk, tv, x, j0, std::true_type());
                }
            }
            if (it + 1 < kt.count) {
                put(it + 1);
                __syncthreads();
            }
        }
    }
    delta = swap_sum(delta);
    if constexpr (SUMMED) {
        __shared__ float s_delta[NW][32];
        if (KS > 1 && h2 == 0) s_delta[w][n] = delta;
        __syncthreads();   // the last tiles are read, too
        if constexpr (KS > 1) {
            delta = 0.f;
#pragma unroll
            for (int y = 0; y < KS; ++y) delta += s_delta[w - wk + y][n];
        }
    }
    if (live && h2 == 0 && wk == 0) p.delta[r0] = delta;
    f32x16 A[MD];
#pragma unroll
    for (int m = 0; m < MD; ++m) A[m] = zero16();
    auto tile = [&](const T* tk, const T* tv, int x, int j0, auto masked) {
        f32x16 s = zero16(), d = zero16();
#pragma unroll
        for (int ks = 0; ks < KD; ++ks) {
            s = mma32(nat32<T>(tk, ST, 32 * x, 16 * ks, n, h2), qf[ks], s);
            d = mma32(nat32<T>(tv, ST, 32 * x, 16 * ks, n, h2), gf[ks], d);
        }
        const Mask mask(row, j0 + 4 * h2, p.window, p.sinks);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const float e = fast_exp2(fmaf(s[r], c, -lse2)) * (d[r] - delta);
            s[r] = !masked.value || mask(result_row(r, 0)) ? e : 0.f;
        }
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            const V8 df = rows16<T>(s, kb);
#pragma unroll
            for (int m = 0; m < MD; ++m) A[m] = mma32(tr32(tk, ST, 32 * x + 16 * kb, 32 * m, lane), df, A[m]);
        }
    };
    fetch(0);
    put(0);
    __syncthreads();
    for (int it = 0; it < kt.count; ++it) {
        if (it + 1 < kt.count) fetch(it + 1);
        const T* tk = tiles + ((it & 1) * 2 * KB + wk * KT) * ST;
        const T* tv = tk + KB * ST;
        if (i0 < len) {
#pragma unroll
            for (int x = 0; x < KT / 32; ++x) {
                const int j0 = kt[it] * KB + wk * KT + 32 * x;
                const Seen se = seen(i0, i0 + 31, j0, j0 + 31, p.window, p.sinks);
                if (se.none) continue;
                if (se.all) tile(tk, tv, x, j0, std::false_type()); else tile(tk, tv, x, j0, std::true_type());
            }
        }
        if (it + 1 < kt.count) {
            put(it + 1);
            __syncthreads();
        }
    }
    if constexpr (KS > 1) {
        static_assert(16 * MD * 4 * 64 * NW <= sizeof(T) * 4 * KB * ST, "room for the join");
        float* const join = reinterpret_cast<float*>(smem) + (size_t)w * 16 * MD * 64 + lane;
        __syncthreads();
        if (wk) {
#pragma unroll
            for (int m = 0; m < MD; ++m)
#pragma unroll
                for (int r = 0; r < 16; ++r) join[(16 * m + r) * 64] = A[m][r];
        }
        __syncthreads();
        if (wk) return;
#pragma unroll
        for (int y = 1; y < KS; ++y)
#pragma unroll
            for (int m = 0; m < MD; ++m)
#pragma unroll
                for (int r = 0; r < 16; ++r) A[m][r] += join[(size_t)(y * 16 * MD + 16 * m + r) * 64];
    }
    if (live) {
        T* out = static_cast<T*>(p.dq) + ((size_t)(ts + row) * p.Hq + h) * D;
#pragma unroll
        for (int m = 0; m < MD; ++m) store_tile<T>(out + 32 * m, A[m], p.scale, h2);
    }
}

// ---------------------------------------------------------------- gradients with respect to k and v

// A workgroup owns KEY_BLOCK keys of one kv head and walks the rows that see
// them, over every query head of the group. P is formed as [rows][keys], a lane
// owning a key: dv^T += dO^T P, dk^T += Q^T dS. Both sums and both operands of 32
// keys would fill a SIMD's registers with one wave, so two waves share the work of
// 32 keys: one holds k, forms P, hands it over through LDS and sums dv; the other
// holds v, forms dP, and dS and dk from it. A tile has 64 rows, two independent
// chains of products a wave; it lies in LDS once, the next one in registers, so
// that two workgroups fit a CU and fill each other's waits. 4,096 rows, 16 and 4 heads,
// d = 128, window 512, 4 sinks, bf16: 104 us, 23 more for the sum of the parts.
// The rows of a block with sinks reach to the end of the sequence: in sequences of
// 2 * sink_rows and more they are cut into equal parts of sink_rows to twice that,
// each a workgroup, summed afterwards in a fixed order.
constexpr int KEY_BLOCK = 64, GRAD_ROWS = 64;

// The parts of every sequence's rows are numbered through: a sequence has those
// from (its first row) / sink_rows up to (its end) / sink_rows, and a block's own
// workgroup takes the first. Batches of short sequences have few numbers or none.
struct SinkParts { int first, count; };
__device__ __forceinline__ SinkParts sink_parts_of(const SwaParams& p, int seq) {
    if (p.sink_parts == 0) return SinkParts{0, 0};
    if (!p.map.cu) return SinkParts{seq * (p.map.T / p.sink_rows), p.map.T / p.sink_rows};
    const int a = seq_offset(p.map, seq), b = max(seq_offset(p.map, seq + 1), a);
    return SinkParts{a / p.sink_rows, b / p.sink_rows - a / p.sink_rows};
}
// the sequence that a number belongs to, and its place there
__device__ __forceinline__ bool sink_part(const SwaParams& p, int v, int& seq, int& part) {
    if (!p.map.cu) {
        seq = v / (p.map.T / p.sink_rows);
    } else {
        int lo = 0, hi = p.map.N - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (seq_offset(p.map, mid) / p.sink_rows <= v) lo = mid; else hi = mid - 1;
        }
        seq = lo;
    }
    const SinkParts sp = sink_parts_of(p, seq);
    part = v - sp.first;
    return part >= 0 && part < sp.count;
}

// Where a part of a block's gradients is kept. Heads of a group in parts: [item][kv
// head][part of the heads], an item being a block or a further part of a block with
// sinks; else [number of the part][kv head][block].
__host__ __device__ inline size_t part_slot(const SwaParams& p, int item, int number, int idx, int hk, int hp) {
    if (p.head_parts > 1) return ((size_t)item * p.Hkv + hk) * p.head_parts + hp;
    return ((size_t)number * p.Hkv + hk) * p.sink_blocks + idx;
}

template <class T, int D> constexpr size_t dkv_lds() {
    return sizeof(T) * 2 * GRAD_ROWS * tile_stride<T>(D) + 8 * GRAD_ROWS + KEY_BLOCK * GRAD_ROWS * 4;
}

template <class T, int D> __global__ void __launch_bounds__(256, 2) swa_dkv_kernel(SwaParams p) {
    constexpr int RT = GRAD_ROWS, NX = RT / 32, NT = 256, KB = KEY_BLOCK, ST = tile_stride<T>(D), KD = D / 16, MD = D / 32;
    using V8 = typename Frag<T>::V;
    extern __shared__ __align__(16) unsigned char smem[];
    lds_poison((uint32_t)dkv_lds<T, D>());
    T* const tq = reinterpret_cast<T*>(smem);   // q and dO of a tile, [RT][ST] each
    T* const tg = tq + RT * ST;
    float* const stats = reinterpret_cast<float*>(tg + RT * ST);   // [lse, delta][RT]
    f32x4* const box = reinterpret_cast<f32x4*>(stats + 2 * RT);   // [32 keys][32 rows][4][lane]: P

    const int tid = threadIdx.x, lane = tid % WAVE, n = lane & 31, h2 = lane >> 5;
    const int w = wave_id() % 2;   // which 32 keys
    const bool grad = wave_id() >= 2;
    // neighbouring key blocks, which read the same rows, on one XCD; parts of
    // blocks with sinks behind them
    const int heads = p.Hkv * p.head_parts, items = p.blocks * heads;
    int hk, item;
    if ((int)blockIdx.x < items) {
        const int e = xcd_remap(blockIdx.x, items);
        hk = e / p.blocks;
        item = e % p.blocks;
    } else {
        hk = (blockIdx.x - items) % heads;
        item = p.blocks + (blockIdx.x - items) / heads;
    }
    const int hp = hk % p.head_parts;
    hk /= p.head_parts;
    const int ga = hp * p.G / p.head_parts, gn = (hp + 1) * p.G / p.head_parts - ga;   // the group's heads taken here
    SeqBlock b;
    int part = 0;
    if (item < p.blocks) {
        if (!seq_block(p.map, KB, item, b)) return;
    } else {   // further parts of the blocks with sinks
        const int e = item - p.blocks;
        if (!sink_part(p, e / p.sink_blocks, b.seq, part) || part == 0) return;
        b.idx = e % p.sink_blocks;
        if (p.map.cu) {
            const int c0 = seq_offset(p.map, b.seq);
            b.t0 = c0;
            b.len = max(seq_offset(p.map, b.seq + 1) - c0, 0);
        } else {
            b.t0 = (long)b.seq * p.map.T;
            b.len = p.map.T;
        }
        b.t0 += (long)b.idx * KB;
        if (b.idx * KB >= b.len) return;
    }
    const int k0 = b.idx * KB, len = b.len;
    const long ts = b.t0 - k0;
    const SinkParts sp = b.idx < p.sink_blocks ? sink_parts_of(p, b.seq) : SinkParts{0, 0};
    const bool sink = sp.count > 1, cut = sink || p.head_parts > 1;
    // rows of this workgroup: the window's, or all to the end, in equal parts
    int ra = k0, rb = k0 < p.sinks ? len : (int)min((long)k0 + KB - 1 + p.window, (long)len);
    if (sink) {
        const int step = ((len - k0 + sp.count - 1) / sp.count + RT - 1) / RT * RT;
        ra = (int)min((long)k0 + (long)part * step, (long)len);
        rb = (int)min((long)ra + step, (long)len);
    }
    const int key = k0 + 32 * w + n;
    const bool live = key < len;
    const float c = p.scale * LOG2E;

    V8 own[KD];   // k or v of the lane's key
    {
        const T* src = static_cast<const T*>(grad ? p.v : p.k) + ((size_t)(ts + (live ? key : 0)) * p.Hkv + hk) * D + 8 * h2;
#pragma unroll
        for (int ks = 0; ks < KD; ++ks) own[ks] = load8<T>(src + 16 * ks, live);
    }
    f32x16 acc[MD];   // dv or dk
#pragma unroll
    for (int m = 0; m < MD; ++m) acc[m] = zero16();

    const int t0 = ra / RT, per = rb > ra ? (rb - 1) / RT - t0 + 1 : 0, count = per * gn;
    const size_t rs = (size_t)p.Hq * D;
    Stage<T, D, RT, NT> sq, sg;
    float stat = 0.f;
    int stat_rows = 0;
    auto fetch = [&](int it) {
        const int h = hk * p.G + ga + it / per, r0 = (t0 + it % per) * RT;
        const size_t at = (size_t)(ts + r0) * p.Hq + h;
        sq.load(static_cast<const T*>(p.q) + at * D, rs, rb - r0, tid);
        sg.load(static_cast<const T*>(p.dO) + at * D, rs, rb - r0, tid);
        // taken as it lies: arithmetic here would wait for the tiles too
        stat_rows = rb - r0;
        if (tid < 2 * RT) stat = (tid < RT ? p.lse : p.delta)[at + (size_t)min(tid % RT, stat_rows - 1) * p.Hq];
    };
    auto put = [&] {
        sq.store(tq, tid);
        sg.store(tg, tid);
        if (tid < 2 * RT) stats[tid] = tid % RT >= stat_rows ? 0.f : tid < RT ? stat * LOG2E : stat;
    };
    f32x4* const mine = box + w * (NX * 4 * WAVE) + lane;
    const float* const sl = stats;
    if (count) {
        fetch(0);
        put();
        __syncthreads();
    }
    for (int it = 0; it < count; ++it) {
        if (it + 1 < count) fetch(it + 1);
        const int i0 = (t0 + it % per) * RT, j0 = k0 + 32 * w;
        const Seen se = seen(i0, i0 + RT - 1, j0, j0 + 31, p.window, p.sinks);
        const bool some = !se.none && i0 + RT - 1 >= ra && i0 < rb;
        f32x16 s[NX];
        if (some) {
            const T* t = grad ? tg : tq;
#pragma unroll
            for (int x = 0; x < NX; ++x) s[x] = zero16();
#pragma unroll
            for (int ks = 0; ks < KD; ++ks)
#pragma unroll
                for (int x = 0; x < NX; ++x) s[x] = mma32(nat32<T>(t, ST, 32 * x, 16 * ks, n, h2), own[ks], s[x]);
            if (!grad) {   // P, and over to the other wave
                auto weigh = [&](auto masked) {
#pragma unroll
                    for (int x = 0; x < NX; ++x) {
                        // row - key and row - ra of the lane's first row; later ones count up
                        const int back = i0 + 32 * x + 4 * h2 - key, from = ra - (i0 + 32 * x + 4 * h2);
#pragma unroll
                        for (int r4 = 0; r4 < 4; ++r4) {
                            const f32x4 l4 = *reinterpret_cast<const f32x4*>(sl + 32 * x + 8 * r4 + 4 * h2);
                            f32x4 e;
#pragma unroll
                            for (int m = 0; m < 4; ++m) {
                                const int o = 8 * r4 + m;
                                const bool in = !masked.value || (o >= from && o >= -back &&
                                                                  (o < p.window - back || key < p.sinks));
                                e[m] = in ? fast_exp2(fmaf(s[x][4 * r4 + m], c, -l4[m])) : 0.f;
                                s[x][4 * r4 + m] = e[m];
                            }
                            mine[(4 * x + r4) * WAVE] = e;
                        }
                    }
                };
                if (se.all && i0 >= ra) weigh(std::false_type()); else weigh(std::true_type());
            }
        }
        __syncthreads();
        if (some) {
            if (grad) {
#pragma unroll
                for (int x = 0; x < NX; ++x)
#pragma unroll
                    for (int r4 = 0; r4 < 4; ++r4) {
                        const f32x4 d4 = *reinterpret_cast<const f32x4*>(sl + RT + 32 * x + 8 * r4 + 4 * h2);
                        const f32x4 e = mine[(4 * x + r4) * WAVE];
                        // where P is zero for a hidden row, dP may be anything
#pragma unroll
                        for (int m = 0; m < 4; ++m)
                            s[x][4 * r4 + m] = e[m] == 0.f ? 0.f : e[m] * (s[x][4 * r4 + m] - d4[m]);
                    }
            }
            const T* t = grad ? tq : tg;
#pragma unroll
            for (int kb = 0; kb < 2 * NX; ++kb) {
                const V8 f = rows16<T>(s[kb / 2], kb % 2);
#pragma unroll
                for (int m = 0; m < MD; ++m) acc[m] = mma32(tr32(t, ST, 16 * kb, 32 * m, lane), f, acc[m]);
            }
        }
        if (it + 1 < count) {
            __syncthreads();
            put();
            __syncthreads();
        }
    }
    float* const part_out = p.part + part_slot(p, item, sp.first + part, b.idx, hk, hp) * (2 * KB * D) + (size_t)grad * (KB * D) +
                            (size_t)(32 * w + n) * D;
    T* const out = static_cast<T*>(grad ? p.dk : p.dv) + ((size_t)(ts + key) * p.Hkv + hk) * D;
#pragma unroll
    for (int m = 0; m < MD; ++m) {
        if (cut) store_tile<float>(part_out + 32 * m, acc[m], 1.f, h2);
        else if (live) store_tile<T>(out + 32 * m, acc[m], grad ? p.scale : 1.f, h2);
    }
}

// the parts of a block, summed in order
template <class T, int D> __global__ void __launch_bounds__(256) swa_part_sum_kernel(SwaParams p) {
    constexpr int KB = KEY_BLOCK;
    lds_poison(0);
    const int hk = blockIdx.y;
    SeqBlock b;
    if (p.head_parts > 1) {
        if (!seq_block(p.map, KB, blockIdx.x, b)) return;
    } else {   // the blocks with sinks of the sequences that are cut
        int part;
        if (!sink_part(p, blockIdx.x / p.sink_blocks, b.seq, part) || part != 0) return;
        b.idx = blockIdx.x % p.sink_blocks;
        if (p.map.cu) {
            const int c0 = seq_offset(p.map, b.seq);
            b.t0 = c0;
            b.len = max(seq_offset(p.map, b.seq + 1) - c0, 0);
        } else {
            b.t0 = (long)b.seq * p.map.T;
            b.len = p.map.T;
        }
        b.t0 += (long)b.idx * KB;
    }
    const SinkParts sp = b.idx < p.sink_blocks ? sink_parts_of(p, b.seq) : SinkParts{0, 0};
    if (sp.count <= 1 && p.head_parts == 1) return;   // written as it was formed
    const int e = 4 * (blockIdx.z * 256 + threadIdx.x);
    if (e >= KB * D || b.idx * KB + e / D >= b.len) return;
    f32x4 v = zero4(), k = zero4();
    const int parts = max(sp.count, 1) * p.head_parts;
    constexpr int U = 8;   // parts in flight (a block with sinks may have dozens)
    for (int q0 = 0; q0 < parts; q0 += U) {
        f32x4 x[U], y[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int part = (q0 + u) / p.head_parts, hp = (q0 + u) % p.head_parts;
            x[u] = y[u] = zero4();
            if (q0 + u >= parts) continue;
            const int item = part ? p.blocks + (sp.first + part) * p.sink_blocks + b.idx : (int)blockIdx.x;
            const float* src = p.part + part_slot(p, item, sp.first + part, b.idx, hk, hp) * (2 * KB * D) + e;
            x[u] = *reinterpret_cast<const f32x4*>(src);
            y[u] = *reinterpret_cast<const f32x4*>(src + KB * D);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            v += x[u];
            k += y[u];
        }
    }
    const size_t to = ((size_t)(b.t0 + e / D) * p.Hkv + hk) * D + e % D;
    store4(static_cast<T*>(p.dv) + to, v);
    store4(static_cast<T*>(p.dk) + to, k * p.scale);
}

// ---------------------------------------------------------------- one token over a cache

struct SwaDecodeParams {
    const void *q, *k, *v;
    void *Kc, *Vc, *o;
    const int32_t* pos;
    float *pm, *pl, *po;   // parts: running maximum (log2), sum, unnormalised o: [N * Hq][splits](, [D])
    int N, Hq, Hkv, G, GC;   // GC: workgroups over a group's heads, 32 each
    int window, sinks, slots, splits, per;   // per: slots of a part
    float scale;
};

// One part of a cache for one kv head: each wave takes every NW-th tile of 32
// slots through LDS of its own (no barrier), the group's query heads side by
// side as the columns. The new token's row is read from k and v, and written to
// its slot by the workgroup whose part holds it. Bound by the cache's bytes: 64 sequences
// of 2,052 slots, 8 kv heads, d = 128, bf16: 88 to 90 us, 5.4 TB/s.
template <class T, int D, int NW> __global__ void __launch_bounds__(64 * NW) swa_decode_kernel(SwaDecodeParams p) {
    constexpr int ST = tile_stride<T>(D), KD = D / 16, MD = D / 32, CPR = D * (int)sizeof(T) / 16, PER = 16 / (int)sizeof(T);
    using V8 = typename Frag<T>::V;
    extern __shared__ __align__(16) unsigned char smem[];
    const uint32_t lds = sizeof(T) * NW * 2 * 32 * ST;
    lds_poison(lds);
    const int tid = threadIdx.x, lane = tid % WAVE, w = wave_id(), n = lane & 31, h2 = lane >> 5;
    T* const tk = reinterpret_cast<T*>(smem) + w * 2 * 32 * ST;
    T* const tv = tk + 32 * ST;
    const int part = blockIdx.x % p.splits, gc = blockIdx.x / p.splits, hk = blockIdx.y, seq = blockIdx.z;
    const int g0 = 32 * gc, gn = min(32, p.G - g0);
    const size_t head0 = (size_t)seq * p.Hq + hk * p.G + g0;
    const int pos = p.pos[seq];
    const int held = pos < 0 ? 0 : (int)min((long)pos + 1, (long)p.slots);
    const int slot = pos < 0 ? -1 : pos < p.sinks ? pos : p.sinks + (pos - p.sinks) % p.window;
    const int a = part * p.per, e = min(a + p.per, held);
    const T* newk = static_cast<const T*>(p.k) + ((size_t)seq * p.Hkv + hk) * D;
    const T* newv = static_cast<const T*>(p.v) + ((size_t)seq * p.Hkv + hk) * D;
    T* Kc = static_cast<T*>(p.Kc) + ((size_t)seq * p.slots * p.Hkv + hk) * D;
    T* Vc = static_cast<T*>(p.Vc) + ((size_t)seq * p.slots * p.Hkv + hk) * D;
    const size_t rs = (size_t)p.Hkv * D;
    if (gc == 0 && slot >= a && slot < e && tid < 2 * CPR) {
        const bool isv = tid >= CPR;
        const int x = (tid - (isv ? CPR : 0)) * PER;
        *reinterpret_cast<uint4*>((isv ? Vc : Kc) + (size_t)slot * rs + x) =
            *reinterpret_cast<const uint4*>((isv ? newv : newk) + x);
    }
    Stage<T, D, 32, 64> rk, rv;
    auto fetch = [&](int j0) {
        rk.load(Kc + (size_t)j0 * rs, rs, e - j0, lane);
        rv.load(Vc + (size_t)j0 * rs, rs, e - j0, lane);
        if (slot >= j0 && slot < min(j0 + 32, e)) {   // the cache's row may not have it yet
#pragma unroll
            for (int m = 0; m < rk.N; ++m) {
                const int x = lane + 64 * m, col = x % CPR * PER;
                if (j0 + x / CPR == slot) {
                    __builtin_memcpy(&rk.r[m], newk + col, 16);
                    __builtin_memcpy(&rv.r[m], newv + col, 16);
                }
            }
        }
    };
    V8 qf[KD];
#pragma unroll
    for (int ks = 0; ks < KD; ++ks)
        qf[ks] = load8<T>(static_cast<const T*>(p.q) + (head0 + (n < gn ? n : 0)) * D + 16 * ks + 8 * h2, n < gn);
    f32x16 O[MD];
#pragma unroll
    for (int m = 0; m < MD; ++m) O[m] = zero16();
    float top = -INFINITY, sum = 0.f;
    const float c = p.scale * LOG2E;
    int j0 = a + 32 * w;
    if (j0 < e) fetch(j0);
    for (; j0 < e; j0 += 32 * NW) {
        // the tile is this wave's own: its reads of the last one are done, its
        // writes are in order before the reads below
        rk.store(tk, lane);
        rv.store(tv, lane);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (j0 + 32 * NW < e) fetch(j0 + 32 * NW);
        f32x16 s = zero16();
#pragma unroll
        for (int ks = 0; ks < KD; ++ks) s = mma32(nat32<T>(tk, ST, 0, 16 * ks, n, h2), qf[ks], s);
        float mt = -INFINITY;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            s[r] = j0 + result_row(r, h2) < e ? s[r] * c : -INFINITY;
            mt = fmaxf(mt, s[r]);
        }
        mt = swap_max(mt);
        const float next = fmaxf(top, mt);
        const float base = next == -INFINITY ? 0.f : next;
        const float f = fast_exp2(top - base);
        top = next;
        sum *= f;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            s[r] = fast_exp2(s[r] - base);
            sum += s[r];
        }
#pragma unroll
        for (int m = 0; m < MD; ++m)
#pragma unroll
            for (int r = 0; r < 16; ++r) O[m][r] *= f;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            const V8 pf = rows16<T>(s, kb);
#pragma unroll
            for (int m = 0; m < MD; ++m) O[m] = mma32(tr32(tv, ST, 16 * kb, 32 * m, lane), pf, O[m]);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    sum = swap_sum(sum);
    // the waves' shares, joined through LDS: o in the tiles' place, [wave][head][D]
    __shared__ float s_top[NW][32], s_sum[NW][32];
    __syncthreads();
    float* so = reinterpret_cast<float*>(smem);
    if (h2 == 0) {
        s_top[w][n] = top;
        s_sum[w][n] = sum;
    }
    if (n < gn) {
#pragma unroll
        for (int m = 0; m < MD; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                *reinterpret_cast<f32x4*>(so + (size_t)(w * 32 + n) * D + 32 * m + 8 * r + 4 * h2) =
                    f32x4{O[m][4 * r], O[m][4 * r + 1], O[m][4 * r + 2], O[m][4 * r + 3]};
    }
    __syncthreads();
    for (int x = tid; x < gn * (D / 4); x += 64 * NW) {
        const int g = x / (D / 4), d = x % (D / 4) * 4;
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int y = 0; y < NW; ++y) m = fmaxf(m, s_top[y][g]);
        const float base = m == -INFINITY ? 0.f : m;
        f32x4 acc = zero4();
#pragma unroll
        for (int y = 0; y < NW; ++y) {
            const float f = fast_exp2(s_top[y][g] - base);
            l += f * s_sum[y][g];
            acc += *reinterpret_cast<const f32x4*>(so + (size_t)(y * 32 + g) * D + d) * f;
        }
        const size_t at = head0 + g;
        if (p.splits == 1) {
            store4(static_cast<T*>(p.o) + at * D + d, pos < 0 ? zero4() : acc * (1.f / l));
        } else {
            *reinterpret_cast<f32x4*>(p.po + (at * p.splits + part) * D + d) = acc;
            if (d == 0) {
                p.pm[at * p.splits + part] = m;
                p.pl[at * p.splits + part] = l;
            }
        }
    }
}

// Joins the parts of one query head: four values a thread, the parts spread over
// the rest of the workgroup (a thread that walked them all would wait for each).
template <class T, int D> __global__ void __launch_bounds__(256) swa_join_kernel(SwaDecodeParams p) {
    lds_poison(0);
    constexpr int CG = D / 4, RG = 256 / CG;
    __shared__ float s_l[RG];
    __shared__ __align__(16) float s_o[RG][D];
    const size_t at = blockIdx.x;
    const int cg = threadIdx.x % CG, rg = threadIdx.x / CG;
    float m = -INFINITY;
    for (int y = 0; y < p.splits; ++y) m = fmaxf(m, p.pm[at * p.splits + y]);
    const float base = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    f32x4 acc = zero4();
    for (int y = rg; y < p.splits; y += RG) {
        const float f = fast_exp2(p.pm[at * p.splits + y] - base);
        l += f * p.pl[at * p.splits + y];
        acc += *reinterpret_cast<const f32x4*>(p.po + (at * p.splits + y) * D + 4 * cg) * f;
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
    store4(static_cast<T*>(p.o) + at * D + 4 * cg, p.pos[at / p.Hq] < 0 ? zero4() : acc * (1.f / l));
}

// ---------------------------------------------------------------- a prompt's keys into a cache

// slot -> the newest position that belongs there; slots that no position of the
// sequence belongs to stay as they are
__global__ void __launch_bounds__(256) swa_fill_kernel(const uint4* __restrict__ k, const uint4* __restrict__ v,
                                                       uint4* __restrict__ Kc, uint4* __restrict__ Vc, SeqMap map,
                                                       int window, int sinks, int slots, int row16) {
    lds_poison(0);
    const int seq = blockIdx.z;
    long t0;
    int len;
    if (map.cu) {
        t0 = seq_offset(map, seq);
        len = max(seq_offset(map, seq + 1) - (int)t0, 0);
    } else {
        t0 = (long)seq * map.T;
        len = map.T;
    }
    for (int slot = blockIdx.x; slot < min(slots, len); slot += gridDim.x) {
        int j = slot;
        if (slot >= sinks) j += (len - 1 - slot) / window * window;
        const size_t from = (size_t)(t0 + j) * row16, to = ((size_t)seq * slots + slot) * row16;
        for (int x = threadIdx.x; x < row16; x += 256) {
            Kc[to + x] = k[from + x];
            Vc[to + x] = v[from + x];
        }
    }
}

// (a launch has fewer than 2^32 threads along x)
template <class K, class P>
hipError_t launch(K kern, size_t x, unsigned y, unsigned z, int threads, size_t lds, hipStream_t st, const P& p) {
    if (x * threads > 0xffffffffu) return hipErrorInvalidConfiguration;
    if (lds > 65536) {
        const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kern, dim3((unsigned)x, y, z), dim3(threads), lds, st, p);
    return hipGetLastError();
}

size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

// Parts of the rows that see a block with sinks: as many rows a part as the window
// gives a block, but at most 64 parts of all blocks of a sequence; none where the
// window covers everything anyway. Forward and gradient of 4,096 rows, 16 and 4
// heads, d = 128, window 512, 4 sinks: 0.339 ms with one walk over all rows for such a
// block, 0.211 in seven parts. More than 2,048 sinks are not cut: each of their blocks
// walks all later rows by itself.
void sink_cut(int T, int N, int window, int sinks, bool packed, SwaParams& p) {
    p.sink_blocks = p.sink_rows = p.sink_parts = 0;
    if (sinks <= 0 || T <= window + KEY_BLOCK) return;
    const int blocks = (int)((std::min((long)sinks, (long)T) + KEY_BLOCK - 1) / KEY_BLOCK), most = 64 / blocks;
    if (most < 2) return;
    const int rows = std::max((window + KEY_BLOCK + 63) / 64 * 64, (T + most - 1) / most);
    if (T / rows < 2) return;
    p.sink_blocks = blocks;
    p.sink_rows = rows;
    p.sink_parts = packed ? T / rows : N * (T / rows);
}

SwaParams make_params(const SwaArgs& a, int NW) {
    SwaParams p{};
    p.q = a.q; p.k = a.k; p.v = a.v; p.o = a.o; p.dO = a.dO; p.lse = a.lse;
    p.out = a.out; p.lse_out = a.lse_out;
    p.dq = a.g_q; p.dk = a.g_k; p.dv = a.g_v;
    p.map = SeqMap{a.cu_seqlens, a.T, a.N};
    p.Hq = a.Hq; p.Hkv = a.Hkv; p.G = a.Hq / a.Hkv;
    p.window = std::min(a.window, a.T);
    p.sinks = std::min(a.sinks, a.T);
    p.scale = a.scale;
    p.HW = heads_together(p.G, NW);
    p.blocks = (int)seq_blocks_bound(a.T, a.N, 32 * NW / p.HW, a.cu_seqlens != nullptr);
    return p;
}

// Waves of a workgroup, in the forward and the gradient of q, that take the same rows: one, where that gives every
// CU a workgroup; else two, or four where the tiles fit LDS, over fewer rows each, as
// long as a row's keys fill the tiles of all. Against workgroups of fewer waves: 1,025
// rows of 6 heads, d = 64, window 100: fp32 14.6 against 19.8 us, bf16 9.6 against 10.2;
// 2,048 rows of 8 heads, d = 128, window 512: 56.8 against 87.1 and 19.1 against 23.0.
// Four where two fill the CUs (1,500 rows of 16 heads, d = 64, window 1024): 43.0
// against 22.6 us. The three gradients of those 1,025 rows against one wave for each: fp32
// 52.6 against 73.2 us, bf16 29.9 against 33.0.
template <class T, int D, int KS, class F> hipError_t split_keys(const SwaArgs& a, F f) {
    constexpr int NW = 4;
    constexpr size_t lds = sizeof(T) * 4 * KS * swa_tile<T>() * tile_stride<T>(D);
    const SwaParams p = make_params(a, NW / KS);
    const size_t wgs = (size_t)p.blocks * (p.Hq / p.HW);
    if constexpr (KS < 4 && 2 * lds <= 160 * 1024)
        if (wgs < 256 && p.window + 32 >= 2 * KS * swa_tile<T>()) return split_keys<T, D, 2 * KS>(a, f);
    return f(p, std::integral_constant<int, KS>(), wgs, 64 * NW, lds);
}

template <class T, int D> hipError_t forward(const SwaArgs& a) {
    return split_keys<T, D, 1>(a, [&](const SwaParams& p, auto ks, size_t wgs, int threads, size_t lds) {
        return launch(swa_fwd_kernel<T, D, 4, ks.value>, wgs, 1, 1, threads, lds, a.stream, p);
    });
}

// workgroups of the gradients of k and v, for a kv head and a part of its heads
long grad_items(const SwaParams& p) { return (long)p.blocks + (long)p.sink_parts * p.sink_blocks; }

// How the gradients of k and v are cut up, and the slots that their parts take.
// Heads of a group are split until there are four workgroups to a CU, two at a
// time: 4,096 rows, 16 and 4 heads, d = 128, window 512, 4 sinks: 0.169 ms whole,
// 0.135 in two parts, 0.109 in four.
size_t grad_parts(int T, int N, int G, int Hkv, int window, int sinks, bool packed, SwaParams& p) {
    sink_cut(T, N, window, sinks, packed, p);
    p.blocks = (int)seq_blocks_bound(T, N, KEY_BLOCK, packed);
    const long items = grad_items(p);
    p.head_parts = (int)std::max(1L, std::min((long)G, (1023 + items * Hkv) / (items * Hkv)));
    if (p.head_parts > 1) return (size_t)items * Hkv * p.head_parts;
    return (size_t)Hkv * p.sink_parts * p.sink_blocks;
}

// rows of a batch
size_t all_rows(int T, int N, bool packed) { return packed ? (size_t)T : (size_t)N * T; }

template <class T, int D> hipError_t backward(const SwaArgs& a) {
    const bool packed = a.cu_seqlens != nullptr;
    char* ws = static_cast<char*>(a.workspace);
    float* const delta = reinterpret_cast<float*>(ws);
    hipError_t e = split_keys<T, D, 1>(a, [&](SwaParams p, auto ks, size_t wgs, int threads, size_t lds) {
        p.delta = delta;
        return launch(swa_dq_kernel<T, D, 4, ks.value>, wgs, 1, 1, threads, lds, a.stream, p);
    });
    if (e != hipSuccess) return e;
    SwaParams p = make_params(a, 1);
    p.delta = delta;
    p.part = reinterpret_cast<float*>(ws + al256(all_rows(a.T, a.N, packed) * a.Hq * 4));
    grad_parts(a.T, a.N, p.G, p.Hkv, p.window, p.sinks, packed, p);
    e = launch(swa_dkv_kernel<T, D>, (size_t)grad_items(p) * p.Hkv * p.head_parts, 1, 1, 256, dkv_lds<T, D>(), a.stream, p);
    if (e != hipSuccess || (p.sink_parts == 0 && p.head_parts == 1)) return e;
    return launch(swa_part_sum_kernel<T, D>, (size_t)(p.head_parts > 1 ? p.blocks : p.sink_parts * p.sink_blocks), p.Hkv,
                  (KEY_BLOCK * D / 4 + 255) / 256, 256, 0, a.stream, p);
}

// Parts of a cache: until two workgroups per CU, each of at least 128 slots. One
// sequence, 4 kv heads, d = 128, bf16, with the launch that joins them: 500 slots 6.9 us
// against 7.4 in one part, 1,000 slots 7.0 against 11.3, 4,096 slots 8.8 against 34.7.
int decode_splits(int N, int Hkv, int gc, int slots) {
    const long wgs = (long)N * Hkv * gc;
    return (int)std::max(1L, std::min((512 + wgs - 1) / wgs, (long)(slots + 127) / 128));
}

template <class T, int D> hipError_t decode(const SwaDecodeArgs& a) {
    constexpr int NW = 4;
    SwaDecodeParams p{};
    p.q = a.q; p.k = a.k; p.v = a.v; p.Kc = a.Kc; p.Vc = a.Vc; p.o = a.o; p.pos = a.pos;
    p.N = a.N; p.Hq = a.Hq; p.Hkv = a.Hkv; p.G = a.Hq / a.Hkv;
    p.GC = (p.G + 31) / 32;
    p.window = a.window; p.sinks = a.sinks; p.slots = a.window + a.sinks;
    p.scale = a.scale;
    p.splits = decode_splits(a.N, a.Hkv, p.GC, p.slots);
    p.per = ((p.slots + p.splits - 1) / p.splits + 31) / 32 * 32;
    const size_t heads = (size_t)a.N * a.Hq;
    p.pm = static_cast<float*>(a.workspace);
    p.pl = p.pm + heads * p.splits;
    p.po = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + al256(heads * p.splits * 8));
    const size_t tiles = sizeof(T) * NW * 2 * 32 * tile_stride<T>(D), join = sizeof(float) * NW * 32 * D;
    hipError_t e = launch(swa_decode_kernel<T, D, NW>, (size_t)p.splits * p.GC, p.Hkv, p.N, 64 * NW, std::max(tiles, join),
                          a.stream, p);
    if (e != hipSuccess || p.splits == 1) return e;
    return launch(swa_join_kernel<T, D>, heads, 1, 1, 256, 0, a.stream, p);
}

#define KDA_SWA_DIM(d, D, ...)                                         \
    [&] {                                                              \
        switch (d) {                                                   \
            case 32: { constexpr int D = 32; return __VA_ARGS__(); }   \
            case 64: { constexpr int D = 64; return __VA_ARGS__(); }   \
            default: { constexpr int D = 128; return __VA_ARGS__(); }  \
        }                                                              \
    }()

}  // namespace

bool swa_grad_fits(int T, int N, int Hq, int Hkv, int window, int sinks, bool packed) {
    if (T <= 0) return true;
    SwaParams p{};
    grad_parts(T, N, Hq / Hkv, Hkv, std::min(window, T), std::min(sinks, T), packed, p);
    return grad_items(p) * Hkv * p.head_parts * 256 <= 0xffffffffL;
}

size_t swa_bwd_workspace_bytes(int T, int N, int Hq, int Hkv, int d, int window, int sinks, bool packed) {
    SwaParams p{};
    const size_t slots = T > 0 ? grad_parts(T, N, Hq / Hkv, Hkv, std::min(window, T), std::min(sinks, T), packed, p) : 0;
    return al256(all_rows(T, N, packed) * Hq * 4 + 1) + slots * 2 * KEY_BLOCK * d * 4;
}

size_t swa_decode_workspace_bytes(int N, int Hq, int Hkv, int d, int window, int sinks) {
    const int splits = decode_splits(N, Hkv, (Hq / Hkv + 31) / 32, window + sinks);
    if (splits == 1) return 256;   // one part writes o itself
    const size_t parts = (size_t)N * Hq * splits;
    return al256(parts * 8) + parts * d * 4;
}

hipError_t launch_swa_fwd(const SwaArgs& a) {
    return KDA_SWA_DIM(a.d, D, [&] { return a.bf16 ? forward<uint16_t, D>(a) : forward<float, D>(a); });
}
hipError_t launch_swa_bwd(const SwaArgs& a) {
    return KDA_SWA_DIM(a.d, D, [&] { return a.bf16 ? backward<uint16_t, D>(a) : backward<float, D>(a); });
}
hipError_t launch_swa_decode(const SwaDecodeArgs& a) {
    return KDA_SWA_DIM(a.d, D, [&] { return a.bf16 ? decode<uint16_t, D>(a) : decode<float, D>(a); });
}

hipError_t launch_swa_cache_fill(const SwaFillArgs& a) {
    const int row16 = (int)((size_t)a.Hkv * a.d * (a.bf16 ? 2 : 4) / 16), slots = a.window + a.sinks;
    hipLaunchKernelGGL(swa_fill_kernel, dim3(std::min({slots, a.T, 1 << 20}), 1, a.N), dim3(256), 0, a.stream, (const uint4*)a.k,
                       (const uint4*)a.v, (uint4*)a.Kc, (uint4*)a.Vc, SeqMap{a.cu_seqlens, a.T, a.N}, a.window, a.sinks,
                       slots, row16);
    return hipGetLastError();
}

}  // namespace kda
