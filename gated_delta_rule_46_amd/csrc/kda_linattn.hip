// Linear attention with a scalar decay per head, over whole sequences and
// backwards:
//
//   S_t = a_t S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t           (S in R^{dk x dv})
//
// Block form. With G_i = a_1..a_i inside a block of C tokens that starts from
// the state S, D_ij = a_{j+1}..a_i (i >= j) and d_j = a_{j+1}..a_C:
//   o_i   = G_i S^T q_i + sum_{j<=i} D_ij (q_i . k_j) v_j
//   S_end = G_C S + sum_j d_j k_j v_j^T
// Every decay factor is a product of decays, never a quotient or a logarithm,
// so zero and negative decays need no special case.
//
// A sequence is cut into segments of several blocks. One launch forms every
// segment's own contribution to the state (all segments in parallel), a second
// combines them in order, elementwise, into the state at each segment start,
// and a third walks every segment from there and writes the outputs: k and v
// are read twice, the states once per segment instead of once per block, and
// nothing longer than a segment is sequential. Short sequences take the third
// launch alone, one segment per sequence.
//
// Backward. With the adjoint G_t = dL/dS_t (G_T = dS_T + q_T dO_T^T,
// G_t = a_{t+1} G_{t+1} + q_t dO_t^T):
//   dq_t = S_t dO_t,  dk_t = G_t v_t,  dv_t = G_t^T k_t,
//   da_t = <S_{t-1}, G_t>,  dS_0 = a_1 G_1.
// The same two launches give S at segment starts and G at segment ends (q, dO
// in place of k, v, in reverse order); in reverse the first keeps what it passes
// at every block as well, so that the last one, block after block of a segment,
// has G at each by one multiplication and addition, and carries S along.
//
// Precision. States and adjoints are held in fp32 wherever they are kept, and a
// token's decayed row enters them as three bf16 numbers (24 mantissa bits: as exact
// as an fp32 sum). bf16 inputs: what enters a product with the inputs is rounded to
// bf16 there, once: decayed scores, states and adjoints. That is as much again as the
// rounding of the results, bf16 themselves: o, dq, dk and dv are off by 2.35e-3 of their
// rms, the decay's gradient by 1.83e-3, where their own rounding makes 1.66e-3 (B = 2, H =
// 16, d = 128, T = 8192 and 4096). Two bf16 numbers an operand would take that away for twice the
// matrix instructions. fp32 inputs: fp32 MFMA throughout.
#include <type_traits>

#include "kda_launch.h"
#include "kda_tiles.h"

namespace kda {

namespace {

struct LinParams {
    const void *q, *k, *v, *gate, *dO;
    const float *S0, *dST;
    void *o, *dq, *dk, *dv, *dgate;
    float *ST, *dS0;
    SeqMap map;
    int H, L;            // heads; tokens per segment (a multiple of the block)
    bool head_gate;      // gate: one fp32 per head, not per token and head
    // [segment][H][dk][dv]: contributions (0: to S, 1: to the adjoint); the scan leaves S
    // at segment starts and the adjoint at segment ends in their place
    float* seg[2];
    float* seg_decay;    // [segment][H]
    // Gradient only, per block: the adjoint at its end as far as it stems from the
    // segment's own tokens, [block][H][dk][dv] (not written for a segment's last
    // block, where it is zero), and the product of the decays between there and
    // the segment's end.
    float *blk, *blk_decay;
};

// Number of the first block (of C tokens) of a segment; a sequence's blocks follow
// each other, numbered as segments are, with C in place of L.
__device__ __forceinline__ long first_block(const LinParams& p, const SeqBlock& b, int C) {
    const long before = p.map.cu ? (b.t0 - (long)b.idx * p.L) / C + b.seq : (long)b.seq * ((p.map.T + C - 1) / C);
    return before + (long)b.idx * (p.L / C);
}

// tokens per block: fp32 tiles are twice as large (64 would not fit the gradient's
// LDS), and fp32 MFMA makes the quadratic part dearer
template <class T> constexpr int lin_block() { return sizeof(T) == 2 ? 64 : 32; }

// ---------------------------------------------------------------- decays of a block

template <int CTRL> __device__ __forceinline__ float dpp_or(float x, float other) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp((int)__float_as_uint(other), (int)__float_as_uint(x), CTRL,
                                                                 0xF, 0xF, false));
}
template <int CTRL> __device__ __forceinline__ float dpp_or_one(float x) { return dpp_or<CTRL>(x, 1.f); }
template <int CTRL> __device__ __forceinline__ double dpp_or_one(double x) {
    const auto u = __builtin_bit_cast(u32x2, x);
    return __builtin_bit_cast(
        double, u32x2{(uint32_t)__builtin_amdgcn_update_dpp(0, (int)u[0], CTRL, 0xF, 0xF, false),
                      (uint32_t)__builtin_amdgcn_update_dpp((int)0x3ff00000, (int)u[1], CTRL, 0xF, 0xF, false)});
}
__device__ __forceinline__ float lane_value(float x, int lane) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(x), lane));
}
__device__ __forceinline__ double lane_value(double x, int lane) {
    const auto u = __builtin_bit_cast(u32x2, x);
    return __builtin_bit_cast(double, u32x2{(uint32_t)__builtin_amdgcn_readlane((int)u[0], lane),
                                            (uint32_t)__builtin_amdgcn_readlane((int)u[1], lane)});
}

template <int C> struct alignas(16) Decays {   // arrays are read four at a time
    static constexpr int DST = 20;   // row stride of diag
    float gam[C];          // a_1..a_i
    float suf[C];          // a_{i+1}..a_C
    float row[C], col[C];  // the same within 16 tokens
    float a[C];
    float diag[C * DST];   // D_ij inside 16 tokens: [i][j % 16]
    float blk[4];          // products over 16 tokens
    float total;
};

template <int C, int D, class R> __device__ __forceinline__ void diag_step(float* row, int il, R a, R& acc) {
    if constexpr (D < 16) {
        if constexpr (D == 1) acc *= a; else acc *= dpp_or_one<0x110 + D - 1>(a);   // row_shr: a_{i-D+1}
        if (il >= D) row[il - D] = (float)acc;
        diag_step<C, D + 1>(row, il, a, acc);
    }
}

// One wave, lane = token, `a` its decay (1 past the sequence's end). Products in R.
template <int C, bool DIAG, class R> __device__ __forceinline__ void products_of_decays(Decays<C>& s, R a, int lane) {
    R p = a, u = a;
    p *= dpp_or_one<0x111>(p); p *= dpp_or_one<0x112>(p); p *= dpp_or_one<0x114>(p); p *= dpp_or_one<0x118>(p);
    u *= dpp_or_one<0x101>(u); u *= dpp_or_one<0x102>(u); u *= dpp_or_one<0x104>(u); u *= dpp_or_one<0x108>(u);
    const R ux = dpp_or_one<0x101>(u);
    R b[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) b[m] = 16 * m < C ? lane_value(p, 16 * m + 15) : R(1);
    const int blk = lane >> 4;
    R pre = 1, post = 1;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        if (m < blk) pre *= b[m];
        if (m > blk) post *= b[m];
    }
    if (lane < C) {
        s.gam[lane] = (float)(pre * p);
        s.suf[lane] = (float)(ux * post);
        s.a[lane] = (float)a;
        if constexpr (DIAG) {
            s.row[lane] = (float)p;
            s.col[lane] = (float)ux;
            float* r = s.diag + lane * Decays<C>::DST;
            const int il = lane & 15;
            r[il] = 1.f;
            R acc = 1;
            diag_step<C, 1>(r, il, a, acc);
        }
    }
    if (lane == 0) {
        s.total = (float)((b[0] * b[1]) * (b[2] * b[3]));
#pragma unroll
        for (int m = 0; m < 4; ++m) s.blk[m] = (float)b[m];
    }
}
// A constant decay's products are formed in 64 bits: in fp32 every one of a power's
// squarings rounds the same way at every block, which had slow heads off by 1e-5 of
// their states after 3,000 tokens. Other decays' roundings differ, and stay in fp32.
template <int C, bool DIAG>
__device__ __forceinline__ void block_decays(Decays<C>& s, const LinParams& p, float a, int lane) {
    if (p.head_gate) products_of_decays<C, DIAG>(s, (double)a, lane);
    else products_of_decays<C, DIAG>(s, a, lane);
}

// D_ij of a 16x16 tile in D-tile order: column i = 16 ti + il, rows j = 16 tj + 4g + r
template <int C>
__device__ __forceinline__ f32x4 tile_decays(const Decays<C>& s, int ti, int tj, int g, int il) {
    const int i = 16 * ti + il;
    if (ti == tj) {
        f32x4 d = *reinterpret_cast<const f32x4*>(s.diag + i * Decays<C>::DST + 4 * g);
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (4 * g + r > il) d[r] = 0.f;
        return d;
    }
    float f = s.row[i];
    for (int m = tj + 1; m < ti; ++m) f *= s.blk[m];
    f32x4 d = *reinterpret_cast<const f32x4*>(s.col + 16 * tj + 4 * g);
    return d * f;
}

// D_{t-1,j} of column t = 16 tt + il, rows j = 16 tj + 4g + r; zero from j = t on
template <int C>
__device__ __forceinline__ f32x4 tile_decays_before(const Decays<C>& s, int tt, int tj, int g, int il) {
    const int t = 16 * tt + il;
    if (tj > tt) return zero4();
    if (tj == tt) {
        f32x4 d = *reinterpret_cast<const f32x4*>(s.diag + max(t - 1, 0) * Decays<C>::DST + 4 * g);
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (4 * g + r >= il) d[r] = 0.f;
        return d;
    }
    float f = il ? s.row[t - 1] : 1.f;
    for (int m = tj + 1; m < tt; ++m) f *= s.blk[m];
    return *reinterpret_cast<const f32x4*>(s.col + 16 * tj + 4 * g) * f;
}

// sum_{j<t} D_{t-1,j} c_j for a lane's token t, c its own term
template <int C> __device__ __forceinline__ float decayed_sum(const Decays<C>& s, float c, int t) {
    float z = c * s.col[t], y = c, a = s.a[t];
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) z += __shfl_xor(z, m, WAVE);   // of 16 tokens, decayed to their end
    // inside 16 tokens: (a, y) of consecutive runs, joined
    y += a * dpp_or<0x111>(y, 0.f); a *= dpp_or_one<0x111>(a);
    y += a * dpp_or<0x112>(y, 0.f); a *= dpp_or_one<0x112>(a);
    y += a * dpp_or<0x114>(y, 0.f); a *= dpp_or_one<0x114>(a);
    y += a * dpp_or<0x118>(y, 0.f);
    y = dpp_or<0x111>(y, 0.f);   // up to t - 1
    float before = 0.f;
#pragma unroll
    for (int m = 0; m < C / 16 - 1; ++m) {
        const float zm = lane_value(z, 16 * m);
        if (m < t / 16) before = before * s.blk[m] + zm;
    }
    return y + (t % 16 ? s.row[t - 1] : 1.f) * before;
}

// A lane's decay as it lies in memory, and its value: apart, so that the load
// can stay in flight over a block's work. Tokens past `n` have decay 1.
template <class T> struct DecayLoad {
    T raw = T(0);
    float head = 1.f;
    int n = 0;
    __device__ __forceinline__ DecayLoad(const LinParams& p, int h) {
        if (p.head_gate) head = static_cast<const float*>(p.gate)[h];
    }
    __device__ __forceinline__ void load(const LinParams& p, long t0, int h, int lane, int tokens) {
        n = tokens;
        if (!p.head_gate) raw = static_cast<const T*>(p.gate)[(size_t)(t0 + min(lane, n - 1)) * p.H + h];
    }
    __device__ __forceinline__ float value(const LinParams& p, int lane) const {
        return lane >= n ? 1.f : p.head_gate ? head : from_el(raw);
    }
};

// 8 factors at kpos(g, .) from position k0 of an LDS array
__device__ __forceinline__ f32x8 factors(const float* s, int k0, int g) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(s + k0 + 4 * g);
    const f32x4 b = *reinterpret_cast<const f32x4*>(s + k0 + 16 + 4 * g);
    return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// x as a sum of PARTS operands of the input type, each the rounding of what the
// ones before leave over
template <class T, int PARTS> __device__ __forceinline__ void split(typename Frag<T>::V (&part)[PARTS], f32x8 x) {
#pragma unroll
    for (int e = 0; e < PARTS; ++e) {
        part[e] = narrow<T>(x);
        if (e + 1 < PARTS) x -= widen(part[e]);
    }
}

// ---------------------------------------------------------------- state walk

// One segment of one head in one direction, from zero: the state's transpose
// (rows dv, columns dk) in accumulators, dk columns split over the waves. Writes
// the segment's contribution and its decay; BLOCKS: in reverse, what it has at
// every block on the way too. Bound by bytes: B = 2, T = 4096, H = 16, d = 128, bf16, both
// directions with BLOCKS 60 us (286 MB, 4.8 TB/s); forward of T = 8192 without 46 us (169 MB,
// 3.7 TB/s).
template <class T, int DK, int DV, int NW, bool BLOCKS>
__global__ void __launch_bounds__(64 * NW) lin_state_kernel(LinParams p) {
    constexpr int C = lin_block<T>(), NT = 64 * NW, NPW = DK / 16 / NW, MT = DV / 16;
    constexpr int SX = tile_stride<T>(DV), SY = tile_stride<T>(DK), PARTS = sizeof(T) == 4 ? 1 : 3;
    using V8 = typename Frag<T>::V;
    extern __shared__ __align__(16) unsigned char smem[];
    lds_poison((uint32_t)(sizeof(Decays<C>) + sizeof(T) * C * (SX + SY)));
    Decays<C>& dec = *reinterpret_cast<Decays<C>*>(smem);
    T* sx = reinterpret_cast<T*>(smem + sizeof(Decays<C>));
    T* sy = sx + C * SX;

    const int tid = threadIdx.x, lane = tid % WAVE, w = wave_id(), g = lane >> 4, il = lane & 15;
    const int h = blockIdx.y, rev = blockIdx.z;
    SeqBlock b;
    if (!seq_block(p.map, p.L, blockIdx.x, b)) return;
    const int nc = (b.n + C - 1) / C;
    const bool keep = BLOCKS && rev;
    const long block0 = keep ? first_block(p, b, C) : 0;
    const size_t at = (size_t)blockIdx.x * p.H + h;
    const T* X = static_cast<const T*>(rev ? p.dO : p.v);
    const T* Y = static_cast<const T*>(rev ? p.q : p.k);
    const size_t rx = (size_t)p.H * DV, ry = (size_t)p.H * DK;

    f32x4 acc[NPW][MT];
#pragma unroll
    for (int x = 0; x < NPW; ++x)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[x][m] = zero4();

    auto put = [&](float* dst) {
#pragma unroll
        for (int x = 0; x < NPW; ++x)
#pragma unroll
            for (int m = 0; m < MT; ++m) store4(dst + (size_t)(16 * (w * NPW + x) + il) * DV + 16 * m + 4 * g, acc[x][m]);
    };
    Stage<T, DV, C, NT> stx;
    Stage<T, DK, C, NT> sty;
    DecayLoad<T> a(p, h);
    float decay = 1.f;
    auto fetch = [&](int step) {
        const int c = rev ? nc - 1 - step : step;
        const long t = b.t0 + (long)c * C;
        const int n = min(C, b.n - c * C);
        stx.load(X + ((size_t)t * p.H + h) * DV, rx, n, tid);
        sty.load(Y + ((size_t)t * p.H + h) * DK, ry, n, tid);
        if (w == 0) a.load(p, t, h, lane, n);
    };
    fetch(0);
    for (int step = 0; step < nc; ++step) {
        const int c = rev ? nc - 1 - step : step;
        if (keep) {
            const size_t to = (size_t)(block0 + c) * p.H + h;
            if (tid == 0) p.blk_decay[to] = decay;
            if (step) put(p.blk + to * (DK * DV));
        }
        if (step) __syncthreads();
        stx.store(sx, tid);
        sty.store(sy, tid);
        if (w == 0) block_decays<C, false>(dec, p, a.value(p, lane), lane);
        __syncthreads();
        if (step + 1 < nc) fetch(step + 1);
        const float tot = dec.total;
        const float* f = rev ? dec.gam : dec.suf;
        decay *= tot;
#pragma unroll
        for (int x = 0; x < NPW; ++x)
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[x][m] *= tot;
#pragma unroll
        for (int ks = 0; ks < C / 32; ++ks) {
            const f32x8 fk = factors(f, 32 * ks, g);
            V8 part[NPW][PARTS];
#pragma unroll
            for (int x = 0; x < NPW; ++x)
                split<T, PARTS>(part[x], widen(frag_tr(sy, SY, 32 * ks, 16 * (w * NPW + x), g, il)) * fk);
            V8 xf[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) xf[m] = frag_tr(sx, SX, 32 * ks, 16 * m, g, il);
#pragma unroll
            for (int e = 0; e < PARTS; ++e)   // no accumulator twice in a row
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int x = 0; x < NPW; ++x) acc[x][m] = mma(xf[m], part[x][e], acc[x][m]);
        }
    }
    put(p.seg[rev] + at * (DK * DV));
    if (tid == 0 && !rev) p.seg_decay[at] = decay;
}

// ---------------------------------------------------------------- scan over segments

// workgroups of a state
__host__ __device__ constexpr int scan_parts(int dkdv) { return (dkdv / 4 + 255) / 256; }

// Elementwise over dk x dv, one (sequence, head) per (blockIdx.x, y); bound by the latency of
// a chain of loads as long as a sequence has segments (eight in flight). Direction 0:
// from the segments' contributions the state at each segment's start, and S_T.
// Direction 1: the adjoint at each one's end, and dS0. In place, in fp32.
__global__ void __launch_bounds__(256) lin_scan_kernel(LinParams p, int dkdv) {
    lds_poison(0);
    const int s = blockIdx.x, h = blockIdx.y, parts = scan_parts(dkdv), rev = blockIdx.z / parts;
    const int e = 4 * (blockIdx.z % parts * 256 + threadIdx.x);
    if (e >= dkdv) return;
    int first, len;
    if (p.map.cu) {
        const int c0 = seq_offset(p.map, s);
        first = c0 / p.L + s;
        len = max(seq_offset(p.map, s + 1) - c0, 0);
    } else {
        len = p.map.T;
        first = s * ((len + p.L - 1) / p.L);
    }
    const int nb = (len + p.L - 1) / p.L;
    const float* init = rev ? p.dST : p.S0;
    float* last = rev ? p.dS0 : p.ST;
    const size_t ends = ((size_t)s * p.H + h) * dkdv + e;
    auto ld4 = [](const float* q) {   // states need element alignment only
        return f32x4{q[0], q[1], q[2], q[3]};
    };
    f32x4 cur = init ? ld4(init + ends) : zero4();
    constexpr int U = 8;   // contributions in flight
    for (int b0 = 0; b0 < nb; b0 += U) {
        f32x4 z[U];
        float d[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (b0 + u >= nb) break;
            const int b = rev ? nb - 1 - (b0 + u) : b0 + u;
            const size_t at = (size_t)(first + b) * p.H + h;
            z[u] = *reinterpret_cast<const f32x4*>(p.seg[rev] + at * dkdv + e);
            d[u] = p.seg_decay[at];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (b0 + u >= nb) break;
            const int b = rev ? nb - 1 - (b0 + u) : b0 + u;
            store4(p.seg[rev] + ((size_t)(first + b) * p.H + h) * dkdv + e, cur);
            cur = cur * d[u] + z[u];
        }
    }
    if (last) {
#pragma unroll
        for (int j = 0; j < 4; ++j) last[ends + j] = cur[j];
    }
}

// ---------------------------------------------------------------- forward outputs

// One segment of one head: the state (rows dk, columns dv) in accumulators, dv
// columns split over the waves; its D tiles are ready A operands of S^T q. B = 2, T =
// 8192, H = 16, d = 128, bf16: 76 us (303 MB, 4.0 TB/s).
// WHOLE: the segment is the whole sequence, from S0 to S_T.
template <class T, int DK, int DV, int NW, bool WHOLE>
__global__ void __launch_bounds__(64 * NW) lin_out_kernel(LinParams p) {
    constexpr int C = lin_block<T>(), NT = 64 * NW, NPW = DV / 16 / NW, MT = DK / 16, CT = C / 16;
    constexpr int KS = tile_cols<T>(DK) / 32, SK = tile_stride<T>(DK), SV = tile_stride<T>(DV), SP = tile_stride<T>(C);
    // a decayed row enters the state, carried over a segment, as one number of the input
    // type (114.6 us), two (117.3) or three, which alone are as exact as the fp32 state (121.5)
    constexpr int PARTS = sizeof(T) == 2 ? 3 : 1;
    using V8 = typename Frag<T>::V;
    extern __shared__ __align__(16) unsigned char smem[];
    lds_poison((uint32_t)(sizeof(Decays<C>) + sizeof(T) * C * (2 * SK + SV + SP)));
    Decays<C>& dec = *reinterpret_cast<Decays<C>*>(smem);
    T* sq = reinterpret_cast<T*>(smem + sizeof(Decays<C>));
    T* sk = sq + C * SK;
    T* sv = sk + C * SK;
    T* sp = sv + C * SV;   // [i][j] decayed scores

    const int tid = threadIdx.x, lane = tid % WAVE, w = wave_id(), g = lane >> 4, il = lane & 15;
    const int h = blockIdx.y;
    SeqBlock b;
    const bool some = seq_block(p.map, p.L, blockIdx.x, b);
    if (!some && !(WHOLE && b.idx == 0)) return;
    const int nc = some ? (b.n + C - 1) / C : 0;
    const size_t ends = ((size_t)b.seq * p.H + h) * (DK * DV);
    const size_t rk = (size_t)p.H * DK, rv = (size_t)p.H * DV;

    Stage<T, DK, C, NT> stq, stk;
    Stage<T, DV, C, NT> stv;
    DecayLoad<T> a(p, h);
    auto fetch = [&](int c) {
        const long t = b.t0 + (long)c * C;
        const int n = min(C, b.n - c * C);
        const size_t r0 = (size_t)t * p.H + h;
        stq.load(static_cast<const T*>(p.q) + r0 * DK, rk, n, tid);
        stk.load(static_cast<const T*>(p.k) + r0 * DK, rk, n, tid);
        stv.load(static_cast<const T*>(p.v) + r0 * DV, rv, n, tid);
        if (w == 0) a.load(p, t, h, lane, n);
    };
    if (nc) fetch(0);
    f32x4 S[NPW][MT];
    auto start = [&](const float* src) {
#pragma unroll
        for (int x = 0; x < NPW; ++x)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    S[x][m][r] = src[(size_t)(16 * m + 4 * g + r) * DV + 16 * (w * NPW + x) + il];
    };
    if constexpr (WHOLE) {
#pragma unroll
        for (int x = 0; x < NPW; ++x)
#pragma unroll
            for (int m = 0; m < MT; ++m) S[x][m] = zero4();
        if (p.S0) start(p.S0 + ends);
    } else {
        start(p.seg[0] + ((size_t)blockIdx.x * p.H + h) * (DK * DV));
    }
    zero_pad_cols<T, DK>(sq, C, tid, NT);
    zero_pad_cols<T, DK>(sk, C, tid, NT);
    for (int c = 0; c < nc; ++c) {
        if (c) __syncthreads();
        stq.store(sq, tid);
        stk.store(sk, tid);
        stv.store(sv, tid);
        if (w == 0) block_decays<C, true>(dec, p, a.value(p, lane), lane);
        __syncthreads();
        if (c + 1 < nc) fetch(c + 1);

        // scores of row tile ti, transposed: rows j, columns i
        for (int ti = w; ti < CT; ti += NW) {
            V8 qf[KS];
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) qf[ks] = frag_nat(sq, SK, 16 * ti + il, 32 * ks, g);
            T* out = sp + (16 * ti + il) * SP + 4 * g;
            for (int tj = 0; tj <= ti; ++tj) {
                f32x4 s = zero4();
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) s = mma(frag_nat(sk, SK, 16 * tj + il, 32 * ks, g), qf[ks], s);
                const f32x4 d = tile_decays<C>(dec, ti, tj, g, il);
#pragma unroll
                for (int r = 0; r < 4; ++r) s[r] = (tj < ti || 4 * g + r <= il) ? s[r] * d[r] : 0.f;
                store4(out + 16 * tj, s);
            }
            if (ti % 2 == 0) store4(out + 16 * (ti + 1), zero4());   // the other half of a 32-deep step
        }
        __syncthreads();

        const int n = min(C, b.n - c * C);
        V8 vf[NPW][C / 32];
#pragma unroll
        for (int x = 0; x < NPW; ++x)
#pragma unroll
            for (int ks = 0; ks < C / 32; ++ks) vf[x][ks] = frag_tr(sv, SV, 32 * ks, 16 * (w * NPW + x), g, il);
        f32x4 acc[NPW][CT];
#pragma unroll
        for (int x = 0; x < NPW; ++x)
#pragma unroll
            for (int tt = 0; tt < CT; ++tt) acc[x][tt] = zero4();
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            V8 sf[NPW];
#pragma unroll
            for (int x = 0; x < NPW; ++x)
                sf[x] = narrow<T>(dtiles_to_frag(S[x][2 * ks], 2 * ks + 1 < MT ? S[x][(2 * ks + 1) % MT] : zero4()));
#pragma unroll
            for (int tt = 0; tt < CT; ++tt) {
                const V8 qf = frag_kpos(sq, SK, 16 * tt + il, 32 * ks, g);
#pragma unroll
                for (int x = 0; x < NPW; ++x) acc[x][tt] = mma(sf[x], qf, acc[x][tt]);
            }
        }
#pragma unroll
        for (int tt = 0; tt < CT; ++tt) {
            const float gi = dec.gam[16 * tt + il];
#pragma unroll
            for (int x = 0; x < NPW; ++x) acc[x][tt] *= gi;
#pragma unroll
            for (int ks = 0; ks <= tt / 2; ++ks) {
                const V8 pf = frag_kpos(sp, SP, 16 * tt + il, 32 * ks, g);
#pragma unroll
                for (int x = 0; x < NPW; ++x) acc[x][tt] = mma(vf[x][ks], pf, acc[x][tt]);
            }
            if (16 * tt + il < n) {
                T* out = static_cast<T*>(p.o) + ((size_t)(b.t0 + c * C + 16 * tt + il) * p.H + h) * DV;
#pragma unroll
                for (int x = 0; x < NPW; x += 2) {
                    if constexpr (NPW > 1) store_pair(out + 16 * (w * NPW + x), acc[x][tt], acc[x + 1][tt], g);
                    else store4(out + 16 * w + 4 * g, acc[x][tt]);
                }
            }
        }
        if (WHOLE || c + 1 < nc) {
            const float tot = dec.total;
#pragma unroll
            for (int x = 0; x < NPW; ++x)
#pragma unroll
                for (int m = 0; m < MT; ++m) S[x][m] *= tot;
#pragma unroll
            for (int ks = 0; ks < C / 32; ++ks) {
                const f32x8 fk = factors(dec.suf, 32 * ks, g);
                V8 part[NPW][PARTS];
#pragma unroll
                for (int x = 0; x < NPW; ++x) split<T, PARTS>(part[x], widen(vf[x][ks]) * fk);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const V8 kf = frag_tr(sk, SK, 32 * ks, 16 * m, g, il);
#pragma unroll
                    for (int x = 0; x < NPW; ++x)
#pragma unroll
                        for (int e = 0; e < PARTS; ++e) S[x][m] = mma(kf, part[x][e], S[x][m]);
                }
            }
        }
    }
    if constexpr (WHOLE) {
        if (p.ST) {
#pragma unroll
            for (int x = 0; x < NPW; ++x)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        p.ST[ends + (size_t)(16 * m + 4 * g + r) * DV + 16 * (w * NPW + x) + il] = S[x][m][r];
        }
    }
}

// ---------------------------------------------------------------- gradients

// The blocks of one segment of one head. With the start state S and the end
// adjoint E of a block:
//   dq_i = G_i S dO_i + sum_{j<=i} D_ij (dO_i . v_j) k_j
//   dk_j = d_j E v_j  + sum_{i>=j} D_ij (dO_i . v_j) q_i
//   dv_j = d_j E^T k_j + sum_{i>=j} D_ij (q_i . k_j) dO_i
// and da_t by its definition as a sum over the pairs (j, i), j < t <= i, of
// their products without a_t: with M_ij = (q_i . k_j)(dO_i . v_j),
//   da_t = sum_{i>=t} D_it R_it,   R_it = sum_{j<t} M_ij D_{t-1,j} + G_{t-1} r_i
//        + d_t (G_{t-1} <S, E> + sum_{j<t} D_{t-1,j} c_j)
// where the start state takes the place of an earlier token (r_i = q_i . S dO_i)
// and the end adjoint that of a later one (c_j = k_j . E v_j). R is one more
// small matrix product, of M and the decays as two bf16 numbers each (bf16 inputs), and
// <S, E> is summed in fp32: with both rounded to one, short sequences had the decay's
// gradient off by up to 2.4 times its own rounding.
// One workgroup fills a CU's LDS: two waves a SIMD, with four barriers a block. Of its 128
// us at B = 2, T = 4096, H = 16, d = 128, bf16 (387 MB of inputs, block adjoints and
// results: 3.0 TB/s) a wave waits for half, and the matrix units are busy for 11%.
template <class T, int DK, int DV, bool DG> struct LinGradTiles {
    // A wave owns one 16-row tile of dk and dv, and so of the state, for a part of a
    // block's tokens (one of TS): bf16 up to 64 columns takes two halves, which form the
    // state twice but keep twice the waves busy. B = 2, T = 4096, H = 16, halves against
    // all tokens: 16 x 16 60 / 85 us, 64 x 64 92 / 113, 128 x 64 133 / 136, 64 x 128
    // 168 / 139, 128 x 128 251 / 185.
    static constexpr int C = lin_block<T>(), NM = (DK > DV ? DK : DV) / 16;
    static constexpr int TS = sizeof(T) == 2 && DV < 128 ? 2 : 1, NW = TS * NM;
    static constexpr int SK = tile_stride<T>(DK), SV = tile_stride<T>(DV), SP = tile_stride<T>(C);
    static constexpr int EROWS = DK < 32 ? 32 : DK;
    Decays<C> dec;
    alignas(16) T q[C * SK], k[C * SK], v[C * SV], dO[C * SV];
    alignas(16) T E[EROWS * SV];
    alignas(16) T p[C * SP], b[C * SP];                       // decayed scores and decayed dO . v, [i][j]
    static constexpr int MN = sizeof(T) == 2 ? 2 : 1;         // M and what its rounding leaves, [i][j]
    alignas(16) T M[MN][DG ? C * SP : 8];
    alignas(16) float r[DG ? NM * C : 4], c[DG ? NM * C : 4], x[NW], da[DG ? C / 16 * C : 4];
};

template <class T, int DK, int DV, bool DG>
__global__ void __launch_bounds__((64 * LinGradTiles<T, DK, DV, DG>::NW)) lin_grad_kernel(LinParams p) {
    using L = LinGradTiles<T, DK, DV, DG>;
    constexpr int C = L::C, NW = L::NW, NT = 64 * NW, CT = C / 16, HT = CT / L::TS, SK = L::SK, SV = L::SV, SP = L::SP;
    constexpr int KSK = tile_cols<T>(DK) / 32, KSV = tile_cols<T>(DV) / 32, KC = C / 32;
    constexpr int KT = DK / 16, VT = DV / 16, PARTS = sizeof(T) == 4 ? 1 : 3;
    using V8 = typename Frag<T>::V;
    extern __shared__ __align__(16) unsigned char smem[];
    lds_poison((uint32_t)sizeof(L));
    L& s = *reinterpret_cast<L*>(smem);

    const int tid0 = threadIdx.x, w = wave_id(), wm = w % L::NM, th = w / L::NM;   // row tile, part of the tokens
    int tid = tid0, lane = tid0 % WAVE, g = lane >> 4, il = lane & 15;
    const int h = blockIdx.y;
    SeqBlock b;
    if (!seq_block(p.map, p.L, blockIdx.x, b)) return;
    const int nc = (b.n + C - 1) / C;
    const long block0 = first_block(p, b, C);
    const size_t rk = (size_t)p.H * DK, rv = (size_t)p.H * DV;

    // what lies beyond a tile's columns, and above the diagonal, stays zero
    zero_pad_cols<T, DK>(s.q, C, tid, NT);
    zero_pad_cols<T, DK>(s.k, C, tid, NT);
    zero_pad_cols<T, DV>(s.v, C, tid, NT);
    zero_pad_cols<T, DV>(s.dO, C, tid, NT);
    zero_pad_cols<T, DV>(s.E, DK, tid, NT);
    if constexpr (DK < 32)   // rows 16..31 of E are contracted over too
        for (int e = tid; e < 16 * SV; e += NT) s.E[16 * SV + e] = T(0);
    for (int e = tid; e < C * SP; e += NT) {
        s.p[e] = s.b[e] = T(0);
        if constexpr (DG)
            for (int y = 0; y < L::MN; ++y) s.M[y][e] = T(0);
    }

    // The state's transpose (rows dv, this wave's columns of dk) in accumulators; its D
    // tiles are ready A operands of S dO. The adjoint on its way to LDS in the same
    // order (EN tiles of a wave): the segment's, held throughout, and a block's own
    // share, loaded ahead for the next block.
    using R4 = typename Raw4<T>::V;
    constexpr int EN = VT < L::TS ? 1 : VT / L::TS;
    const int x0 = th * EN, erow = 16 * wm + il;
    const bool stages = wm < KT && x0 < VT;
    const size_t seg = ((size_t)blockIdx.x * p.H + h) * (DK * DV), own = (size_t)erow * DV + 4 * g;
    f32x4 S[VT], segE[EN], locE[EN];
#pragma unroll
    for (int x = 0; x < VT; ++x) {
        S[x] = zero4();
        if (wm < KT) S[x] = *reinterpret_cast<const f32x4*>(p.seg[0] + seg + own + 16 * x);
    }
#pragma unroll
    for (int x = 0; x < EN; ++x) {
        segE[x] = zero4();
        if (stages) segE[x] = *reinterpret_cast<const f32x4*>(p.seg[1] + seg + own + 16 * (x0 + x));
    }

    Stage<T, DK, C, NT> stq, stk;
    Stage<T, DV, C, NT> stv, sto;
    DecayLoad<T> a(p, h);
    float preE = 1.f;
    // The next block's loads, in three parts between the phases of this one: a
    // wave waits where the memory pipe is full, and registers are freest last.
    auto fetch_qk = [&](int c) {
        const long t = b.t0 + (long)c * C;
        const size_t r0 = (size_t)t * p.H + h;
        const int n = min(C, b.n - c * C);
        stq.load(static_cast<const T*>(p.q) + r0 * DK, rk, n, tid);
        stk.load(static_cast<const T*>(p.k) + r0 * DK, rk, n, tid);
        if (w == 0) a.load(p, t, h, lane, n);
    };
    auto fetch_vo = [&](int c) {
        const size_t r0 = (size_t)(b.t0 + (long)c * C) * p.H + h;
        const int n = min(C, b.n - c * C);
        stv.load(static_cast<const T*>(p.v) + r0 * DV, rv, n, tid);
        sto.load(static_cast<const T*>(p.dO) + r0 * DV, rv, n, tid);
    };
    auto fetch_state = [&](int c) {
        const size_t bs = (size_t)(block0 + c) * p.H + h;
#pragma unroll
        for (int x = 0; x < EN; ++x) {
            locE[x] = zero4();
            if (stages && c + 1 < nc)
                locE[x] = *reinterpret_cast<const f32x4*>(p.blk + bs * (DK * DV) + own + 16 * (x0 + x));
        }
        preE = p.blk_decay[bs];
    };
    fetch_qk(0);
    fetch_vo(0);
    fetch_state(0);
    for (int c = 0; c < nc; ++c) {
        tid = here(tid0);
        lane = tid % WAVE;
        g = lane >> 4;
        il = lane & 15;
        const long t0 = b.t0 + (long)c * C;
        const int n = min(C, b.n - c * C);
        const size_t r0 = (size_t)t0 * p.H + h;
        if (c) __syncthreads();   // the last block's reads are done, its decays' too
        stq.store(s.q, tid);
        stk.store(s.k, tid);
        stv.store(s.v, tid);
        sto.store(s.dO, tid);
        // the adjoint at this block: the segment's, decayed, and its own tokens' share
        float xe = 0.f;
        if (stages) {
#pragma unroll
            for (int x = 0; x < EN; ++x) {
                const f32x4 e = segE[x] * preE + locE[x];
                store4(s.E + (16 * wm + il) * SV + 16 * (x0 + x) + 4 * g, e);
                if constexpr (DG) {
                    f32x4 y = S[x];
                    if constexpr (L::TS == 2) {   // the wave's half, without an index into registers
                        const f32x4 z = raw_here(S[(x + EN) % VT]);
#pragma unroll
                        for (int r = 0; r < 4; ++r) y[r] = th ? z[r] : y[r];
                    }
                    xe += (e[0] * y[0] + e[1] * y[1]) + (e[2] * y[2] + e[3] * y[3]);
                }
            }
        }
        if constexpr (DG) {
            xe = wave_sum(xe);
            if (lane == 0) s.x[w] = xe;
        }
        if (w == 0) block_decays<C, true>(s.dec, p, a.value(p, lane), lane);
        __syncthreads();
        if (c + 1 < nc) fetch_qk(c + 1);

        // pairs of row tiles, transposed: rows j, columns i
        for (int e = w; e < CT * (CT + 1) / 2; e += NW) {
            int ti = 0, tj = e;
            while (tj > ti) { tj -= ti + 1; ++ti; }
            f32x4 x = zero4(), y = zero4();
#pragma unroll
            for (int ks = 0; ks < KSK; ++ks)
                x = mma(frag_nat(s.k, SK, 16 * tj + il, 32 * ks, g), frag_nat(s.q, SK, 16 * ti + il, 32 * ks, g), x);
#pragma unroll
            for (int ks = 0; ks < KSV; ++ks)
                y = mma(frag_nat(s.v, SV, 16 * tj + il, 32 * ks, g), frag_nat(s.dO, SV, 16 * ti + il, 32 * ks, g), y);
            const f32x4 d = tile_decays<C>(s.dec, ti, tj, g, il);
            const int to = (16 * ti + il) * SP + 16 * tj + 4 * g;
            f32x4 m = zero4();
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const bool in = tj < ti || 4 * g + r <= il;
                m[r] = in ? x[r] * y[r] : 0.f;
                x[r] = in ? x[r] * d[r] : 0.f;
                y[r] = in ? y[r] * d[r] : 0.f;
            }
            store4(s.p + to, x);
            store4(s.b + to, y);
            if constexpr (DG) {
                store4(s.M[0] + to, m);
                if constexpr (L::MN == 2) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) m[r] -= (float)(__bf16)m[r];
                    store4(s.M[1] + to, m);
                }
            }
        }

        // products with the boundary states, rounded to the input type here
        f32x4 aq[HT], ak[HT], av[HT];
#pragma unroll
        for (int tt = 0; tt < HT; ++tt) aq[tt] = ak[tt] = av[tt] = zero4();
        if (wm < KT) {
#pragma unroll
            for (int ks = 0; ks < KSV; ++ks) {
                const V8 sf = narrow<T>(dtiles_to_frag(S[2 * ks], 2 * ks + 1 < VT ? S[(2 * ks + 1) % VT] : zero4()));
                const V8 ef = frag_kpos(s.E, SV, 16 * wm + il, 32 * ks, g);
#pragma unroll
                for (int tt = 0; tt < HT; ++tt) {
                    const int i = 16 * (HT * th + tt) + il;
                    aq[tt] = mma(sf, frag_kpos(s.dO, SV, i, 32 * ks, g), aq[tt]);
                    ak[tt] = mma(ef, frag_kpos(s.v, SV, i, 32 * ks, g), ak[tt]);
                }
            }
            if constexpr (DG) {
#pragma unroll
                for (int tt = 0; tt < HT; ++tt) {
                    const int i = 16 * (HT * th + tt) + il;
                    const f32x4 x = aq[tt] * values(*reinterpret_cast<const R4*>(s.q + i * SK + 16 * wm + 4 * g));
                    const f32x4 y = ak[tt] * values(*reinterpret_cast<const R4*>(s.k + i * SK + 16 * wm + 4 * g));
                    float rr = (x[0] + x[1]) + (x[2] + x[3]), cc = (y[0] + y[1]) + (y[2] + y[3]);
                    rr += __shfl_xor(rr, 16, WAVE);
                    rr += __shfl_xor(rr, 32, WAVE);
                    cc += __shfl_xor(cc, 16, WAVE);
                    cc += __shfl_xor(cc, 32, WAVE);
                    if (g == 0) {
                        s.r[wm * C + i] = rr;
                        s.c[wm * C + i] = cc;
                    }
                }
            }
        }
        if (wm < VT) {
#pragma unroll
            for (int ks = 0; ks < KSK; ++ks) {
                const V8 ef = frag_tr(s.E, SV, 32 * ks, 16 * wm, g, il);
#pragma unroll
                for (int tt = 0; tt < HT; ++tt) av[tt] = mma(ef, frag_kpos(s.k, SK, 16 * (HT * th + tt) + il, 32 * ks, g), av[tt]);
            }
        }
#pragma unroll
        for (int tt = 0; tt < HT; ++tt) {
            const int i = 16 * (HT * th + tt) + il;
            const float gi = s.dec.gam[i], di = s.dec.suf[i];
            aq[tt] *= gi;
            ak[tt] *= di;
            av[tt] *= di;
        }
        __syncthreads();
        if (c + 1 < nc) fetch_vo(c + 1);

        // products inside the block; a 32-deep step on the wrong side of the
        // diagonal is skipped
#pragma unroll
        for (int ks = 0; ks < KC; ++ks) {
            V8 kf, qf, of;
            if (wm < KT) {
                kf = frag_tr(s.k, SK, 32 * ks, 16 * wm, g, il);
                qf = frag_tr(s.q, SK, 32 * ks, 16 * wm, g, il);
            }
            if (wm < VT) of = frag_tr(s.dO, SV, 32 * ks, 16 * wm, g, il);
#pragma unroll
            for (int tt = 0; tt < HT; ++tt) {
                const int t = HT * th + tt;
                if (ks <= t / 2 && wm < KT) aq[tt] = mma(kf, frag_kpos(s.b, SP, 16 * t + il, 32 * ks, g), aq[tt]);
                if (ks >= t / 2 && wm < KT) ak[tt] = mma(qf, frag_tr(s.b, SP, 32 * ks, 16 * t, g, il), ak[tt]);
                if (ks >= t / 2 && wm < VT) av[tt] = mma(of, frag_tr(s.p, SP, 32 * ks, 16 * t, g, il), av[tt]);
            }
        }
#pragma unroll
        for (int tt = 0; tt < HT; ++tt) {
            const int i = 16 * (HT * th + tt) + il;
            if (i >= n) continue;
            const size_t row = r0 + (size_t)i * p.H;
            if (wm < KT) {
                store4(static_cast<T*>(p.dq) + row * DK + 16 * wm + 4 * g, aq[tt]);
                store4(static_cast<T*>(p.dk) + row * DK + 16 * wm + 4 * g, ak[tt]);
            }
            if (wm < VT) store4(static_cast<T*>(p.dv) + row * DV + 16 * wm + 4 * g, av[tt]);
        }

        // the state at the next block
        if (c + 1 < nc && wm < KT) {
            constexpr int U = VT < 4 ? VT : 4;   // no accumulator twice in a row
            const float tot = s.dec.total;
#pragma unroll
            for (int x = 0; x < VT; ++x) S[x] *= tot;
#pragma unroll
            for (int ks = 0; ks < KC; ++ks) {
                V8 part[PARTS], vf[U];
                split<T, PARTS>(part, widen(frag_tr(s.k, SK, 32 * ks, 16 * wm, g, il)) * factors(s.dec.suf, 32 * ks, g));
#pragma unroll
                for (int x = 0; x < VT; x += U) {
#pragma unroll
                    for (int u = 0; u < U; ++u) vf[u] = frag_tr(s.v, SV, 32 * ks, 16 * (x + u), g, il);
#pragma unroll
                    for (int e = 0; e < PARTS; ++e)
#pragma unroll
                        for (int u = 0; u < U; ++u) S[x + u] = mma(vf[u], part[e], S[x + u]);
                }
            }
        }
        if constexpr (!DG)
            if (c + 1 < nc) fetch_state(c + 1);
        if constexpr (DG) {
            // R tiles: rows i, columns t
            for (int e = w; e < CT * (CT + 1) / 2; e += NW) {
                int ti = 0, tt = e;
                while (tt > ti) { tt -= ti + 1; ++ti; }
                const int t = 16 * tt + il;
                f32x4 R = zero4();
                for (int ks = 0; ks <= tt / 2; ++ks) {
                    V8 d[L::MN];
                    split<T, L::MN>(d, dtiles_to_frag(tile_decays_before<C>(s.dec, tt, 2 * ks, g, il),
                                                      tile_decays_before<C>(s.dec, tt, 2 * ks + 1, g, il)));
                    const V8 m = frag_kpos(s.M[0], SP, 16 * ti + il, 32 * ks, g);
                    R = mma(m, d[0], R);
                    if constexpr (L::MN == 2) {
                        R = mma(m, d[1], R);
                        R = mma(frag_kpos(s.M[1], SP, 16 * ti + il, 32 * ks, g), d[0], R);
                    }
                }
                f32x4 ri = zero4();
#pragma unroll
                for (int m = 0; m < KT; ++m) ri += *reinterpret_cast<const f32x4*>(s.r + m * C + 16 * ti + 4 * g);
                R += ri * (t ? s.dec.gam[t - 1] : 1.f);
                float mid = 1.f;
                for (int m = tt + 1; m < ti; ++m) mid *= s.dec.blk[m];
                if (tt < ti) mid *= s.dec.col[t];
                float sum = 0.f;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = 16 * ti + 4 * g + r;
                    const float d = tt < ti ? s.dec.row[i] * mid : 4 * g + r >= il ? s.dec.diag[i * Decays<C>::DST + il] : 0.f;
                    if (tt < ti || 4 * g + r >= il) sum += R[r] * d;
                }
                sum += __shfl_xor(sum, 16, WAVE);
                sum += __shfl_xor(sum, 32, WAVE);
                if (g == 0) s.da[ti * C + t] = sum;
            }
            if (c + 1 < nc) fetch_state(c + 1);
            __syncthreads();
            if (w == NW - 1) {
                const int t = lane % C;   // C = 32: the upper lanes repeat the lower ones
                float c0 = 0.f, X = 0.f;
                for (int m = 0; m < KT; ++m) c0 += s.c[m * C + t];
                for (int m = 0; m < NW; ++m) X += s.x[m];
                float acc = s.dec.suf[t] * (X * (t ? s.dec.gam[t - 1] : 1.f) + decayed_sum<C>(s.dec, c0, t));
                for (int m = t / 16; m < CT; ++m) acc += s.da[m * C + t];
                if (lane < n) store1(static_cast<T*>(p.dgate) + (size_t)(t0 + lane) * p.H + h, acc);
            }
        }
    }
}

// ---------------------------------------------------------------- decode

// S' = a S + k v^T, o = S'^T q = a (S^T q) + (k . q) v, the state streamed once in
// and once out, all of it in flight at once: one workgroup a head, 16 bytes a thread
// and load. Bound by those bytes: 256 sequences of 32 heads, 128 x 128, 0.211 ms, 5.1 TB/s
// of state (three states in turn; 0.202 ms on one, part of which the last-level cache
// still holds: the stores go past it). One head over four workgroups, a quarter of its columns each: 3.3 against 3.4 us
// at 16 heads, 6.3 against 5.5 at 256, so it is not done.
template <class T, int DK, int DV, int NT>
__global__ void __launch_bounds__(NT) lin_decode_kernel(const T* __restrict__ q, const T* __restrict__ k,
                                                        const T* __restrict__ v, const void* __restrict__ gate,
                                                        float* __restrict__ S, T* __restrict__ o, int H, int head_gate) {
    constexpr int CG = DV / 4, RG = NT / CG, RPT = DK / RG, NW = NT / WAVE;
    static_assert(NT % WAVE == 0 && DK % RG == 0 && RPT >= 1, "decode tiling");
    lds_poison(0);
    __shared__ float s_k[DK], s_q[DK], s_kq[NW];
    __shared__ __align__(16) float s_v[DV], s_red[NW][DV];   // read and written four at a time
    const size_t pair = blockIdx.x;
    const int t = threadIdx.x, cg = t % CG, rg = t / CG, lane = t % WAVE, w = t / WAVE;
    float kq = 0.f;
    for (int e = t; e < DK; e += NT) {
        const float kv = ld_in(k + pair * DK + e), qv = ld_in(q + pair * DK + e);
        s_k[e] = kv;
        s_q[e] = qv;
        kq += kv * qv;
    }
    for (int e = t; e < DV; e += NT) s_v[e] = ld_in(v + pair * DV + e);
    const float a = head_gate ? static_cast<const float*>(gate)[pair % H] : ld_in(static_cast<const T*>(gate) + pair);
    f32x4* Sp = reinterpret_cast<f32x4*>(S + pair * DK * DV);
    const size_t rs = DV / 4;
    f32x4 sv[RPT];
#pragma unroll
    for (int m = 0; m < RPT; ++m) sv[m] = Sp[(size_t)(rg + RG * m) * rs + cg];
    kq = wave_sum(kq);
    if (lane == 0) s_kq[w] = kq;
    __syncthreads();
    const f32x4 vv = *reinterpret_cast<const f32x4*>(s_v + 4 * cg);
    f32x4 y = zero4();
#pragma unroll
    for (int m = 0; m < RPT; ++m) {
        const int r = rg + RG * m;
        y += sv[m] * s_q[r];
        const f32x4 nv = sv[m] * a + vv * s_k[r];
        __builtin_nontemporal_store(nv, Sp + (size_t)r * rs + cg);
    }
#pragma unroll
    for (int off = CG; off < WAVE; off <<= 1)
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] += __shfl_xor(y[j], off, WAVE);
    if (lane < CG) *reinterpret_cast<f32x4*>(&s_red[w][4 * cg]) = y;
    __syncthreads();
    if (t < DV) {
        float acc = 0.f, dot = 0.f;
#pragma unroll
        for (int m = 0; m < NW; ++m) {
            acc += s_red[m][t];
            dot += s_kq[m];
        }
        store1(o + pair * DV + t, a * acc + dot * s_v[t]);
    }
}

size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

// Tokens per segment: as few segments as give every CU two workgroups, or one in
// the gradient, of which a CU's LDS holds one (over 32 columns). B = 2, T = 4096, H =
// 16: gradient with 256, 512 and 1,024 segments over all heads 185, 217 and 280 us at
// 128 x 128, 92, 99 and 113 at 64 x 64, 82, 55 and 58 at 32 x 32; forward at T = 8192,
// 128 x 128: 133, 121, 150 us.
int segment_tokens(int T, int N, int H, int dk, int dv, bool packed, bool grad) {
    const long tokens = packed ? T : (long)T * N;
    const long want = tokens * H / (grad && (dk > 32 || dv > 32) ? 256 : 512);
    long L = (want + 63) / 64 * 64;
    if (L < 64) L = 64;
    const long whole = ((long)T + 63) / 64 * 64;
    return (int)(L < whole ? L : (whole > 0 ? whole : 64));
}
// Short sequences whole, in one launch. B = 4, H = 16, d = 128: 14.2 against 23.6 us in
// segments at 128 tokens, 21.7 against 29.2 at 256, 30.5 against 33.5 at 384, 39.3 against
// 39.3 at 512. The rule looks at the length alone: where sequences by heads fill the card
// by themselves (512 and more), whole ones would be faster at any length (B = 32, H = 16, T =
// 2048: 265 us against 409), since a segment is a sequence there and is walked twice.
bool whole_sequences(int T) { return T <= 256; }

struct LinWorkspace {
    size_t seg[2], decay, blk, blk_decay, total;
};
LinWorkspace workspace_layout(int T, int N, int H, int dk, int dv, bool packed, bool bf16, bool grad, int L) {
    const size_t segs = (size_t)seq_blocks_bound(T, N, L, packed) * H, state = (size_t)dk * dv;
    const size_t blocks = (size_t)seq_blocks_bound(T, N, bf16 ? lin_block<uint16_t>() : lin_block<float>(), packed) * H;
    LinWorkspace w{};
    size_t at = 0;
    auto take = [&](size_t bytes) { const size_t r = at; at += al256(bytes); return r; };
    w.seg[0] = take(segs * state * 4);
    w.decay = take(segs * 4);
    if (grad) {
        w.seg[1] = take(segs * state * 4);
        w.blk = take(blocks * state * 4);
        w.blk_decay = take(blocks * 4);
    }
    w.total = at;
    return w;
}

// A launch has fewer than 2^32 threads along x. The sizes that the calls accept
// (N * (T + 128) < 2^31) give fewer than 2^24 segments, at most 512 more than
// sequences, so that only the gradient's 512 and 1,024 threads can exceed it.
template <class K, class... A>
hipError_t launch(K kern, size_t x, unsigned y, unsigned z, int threads, size_t lds, hipStream_t stream, A... args) {
    if (x * threads > 0xffffffffu) return hipErrorInvalidConfiguration;
    if (lds > 65536) {
        const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kern, dim3((unsigned)x, y, z), dim3(threads), lds, stream, args...);
    return hipGetLastError();
}

template <class T, int DK, int DV, bool BLOCKS>
hipError_t launch_state(const LinParams& p, int segs, int dirs, hipStream_t st) {
    constexpr int NW = DK / 16 < 4 ? DK / 16 : 4, C = lin_block<T>();
    return launch(lin_state_kernel<T, DK, DV, NW, BLOCKS>, segs, p.H, dirs, 64 * NW,
                  sizeof(Decays<C>) + sizeof(T) * C * (tile_stride<T>(DK) + tile_stride<T>(DV)), st, p);
}

template <class T, int DK, int DV, bool WHOLE> hipError_t launch_out(const LinParams& p, int segs, hipStream_t st) {
    constexpr int NW = DV / 16 < 4 ? DV / 16 : 4, C = lin_block<T>();
    return launch(lin_out_kernel<T, DK, DV, NW, WHOLE>, segs, p.H, 1, 64 * NW,
                  sizeof(Decays<C>) + sizeof(T) * C * (2 * tile_stride<T>(DK) + tile_stride<T>(DV) + tile_stride<T>(C)), st,
                  p);
}

template <class T, int DK, int DV> hipError_t forward(LinParams p, const LinArgs& a) {
    const bool packed = p.map.cu != nullptr;
    if (p.map.T > 0 && whole_sequences(p.map.T)) {
        p.L = (p.map.T + 63) / 64 * 64;
        return launch_out<T, DK, DV, true>(p, (int)seq_blocks_bound(p.map.T, p.map.N, p.L, packed), a.stream);
    }
    const int segs = (int)seq_blocks_bound(p.map.T, p.map.N, p.L, packed);
    hipError_t e = hipSuccess;
    if (p.map.T > 0) e = launch_state<T, DK, DV, false>(p, segs, 1, a.stream);
    if (e != hipSuccess) return e;
    e = launch(lin_scan_kernel, p.map.N, p.H, scan_parts(DK * DV), 256, 0, a.stream, p, DK * DV);
    if (e != hipSuccess || p.map.T == 0) return e;
    return launch_out<T, DK, DV, false>(p, segs, a.stream);
}

template <class T, int DK, int DV> hipError_t backward(const LinParams& p, const LinArgs& a) {
    const bool packed = p.map.cu != nullptr;
    const int segs = (int)seq_blocks_bound(p.map.T, p.map.N, p.L, packed);
    hipError_t e = hipSuccess;
    if (p.map.T > 0) e = launch_state<T, DK, DV, true>(p, segs, 2, a.stream);
    if (e != hipSuccess) return e;
    e = launch(lin_scan_kernel, p.map.N, p.H, 2 * scan_parts(DK * DV), 256, 0, a.stream, p, DK * DV);
    if (e != hipSuccess || p.map.T == 0) return e;
    auto go = [&](auto kern, auto dg) {
        using L = LinGradTiles<T, DK, DV, dg.value>;
        return launch(kern, segs, p.H, 1, 64 * L::NW, sizeof(L), a.stream, p);
    };
    if (p.head_gate) return go(lin_grad_kernel<T, DK, DV, false>, std::false_type());
    return go(lin_grad_kernel<T, DK, DV, true>, std::true_type());
}

template <class T, int DK, int DV> hipError_t decode(const LinDecodeArgs& a) {
    constexpr int NT = lin_decode_threads(DK, DV);
    return launch(lin_decode_kernel<T, DK, DV, NT>, (size_t)a.N * a.H, 1, 1, NT, 0, a.stream, (const T*)a.q, (const T*)a.k,
                  (const T*)a.v, a.gate, a.S, (T*)a.o, a.H, (int)a.head_gate);
}

LinParams make_params(const LinArgs& a) {
    LinParams p{};
    p.q = a.q; p.k = a.k; p.v = a.v; p.gate = a.gate; p.dO = a.dO;
    p.S0 = a.S0; p.dST = a.dST;
    p.o = a.o; p.dq = a.g_q; p.dk = a.g_k; p.dv = a.g_v; p.dgate = a.g_gate;
    p.ST = a.S_T; p.dS0 = a.g_S0;
    p.map = SeqMap{a.cu_seqlens, a.T, a.N};
    p.H = a.H;
    p.head_gate = a.head_gate;
    const bool packed = a.cu_seqlens != nullptr, grad = a.dO != nullptr || a.g_q != nullptr;
    p.L = segment_tokens(a.T, a.N, a.H, a.dk, a.dv, packed, grad);
    const LinWorkspace w = workspace_layout(a.T, a.N, a.H, a.dk, a.dv, packed, a.bf16, grad, p.L);
    char* base = static_cast<char*>(a.workspace);
    for (int d = 0; d < 2; ++d) p.seg[d] = reinterpret_cast<float*>(base + w.seg[d]);
    p.blk = reinterpret_cast<float*>(base + w.blk);
    p.blk_decay = reinterpret_cast<float*>(base + w.blk_decay);
    p.seg_decay = reinterpret_cast<float*>(base + w.decay);
    return p;
}

}  // namespace

size_t lin_workspace_bytes(int B, int H, int T, int dk, int dv, bool packed, int N, bool bf16, bool grad) {
    if (!packed) N = B;
    if (!grad && T > 0 && whole_sequences(T)) return 256;
    const size_t n = workspace_layout(T, N, H, dk, dv, packed, bf16, grad, segment_tokens(T, N, H, dk, dv, packed, grad)).total;
    return n ? n : 256;
}

bool lin_grad_fits(int T, int N, int H, int dk, int dv, bool packed, bool bf16) {
    const long segs = seq_blocks_bound(T, N, segment_tokens(T, N, H, dk, dv, packed, true), packed);
    const long threads = KDA_SWITCH_DIM(dk, DK, [&] {
        return KDA_SWITCH_DIM(dv, DV, [&] {
            return 64L * (bf16 ? LinGradTiles<uint16_t, DK, DV, true>::NW : LinGradTiles<float, DK, DV, true>::NW);
        });
    });
    return segs * threads <= 0xffffffffL;
}

hipError_t launch_lin_fwd(const LinArgs& a) {
    const LinParams p = make_params(a);
    return KDA_SWITCH_DIM(a.dk, DK, [&] {
        return KDA_SWITCH_DIM(a.dv, DV, [&] {
            return a.bf16 ? forward<uint16_t, DK, DV>(p, a) : forward<float, DK, DV>(p, a);
        });
    });
}

hipError_t launch_lin_bwd(const LinArgs& a) {
    const LinParams p = make_params(a);
    return KDA_SWITCH_DIM(a.dk, DK, [&] {
        return KDA_SWITCH_DIM(a.dv, DV, [&] {
            return a.bf16 ? backward<uint16_t, DK, DV>(p, a) : backward<float, DK, DV>(p, a);
        });
    });
}

hipError_t launch_lin_decode(const LinDecodeArgs& a) {
    return KDA_SWITCH_DIM(a.dk, DK, [&] {
        return KDA_SWITCH_DIM(a.dv, DV, [&] {
            return a.bf16 ? decode<uint16_t, DK, DV>(a) : decode<float, DK, DV>(a);
        });
    });
}

}  // namespace kda
