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
// in place of k, v, in reverse order); a walk stores both at every block, and
// the last launch takes all blocks in parallel.
//
// Precision. Products of inputs are exact in fp32. bf16 inputs: scores, states
// and scaled rows enter the next product rounded to bf16, which moves o and the
// gradients (bf16 themselves) by less than their own rounding; sums into the
// final states S_T and dS_0, which are fp32, take the scaled rows as three bf16
// numbers (24 mantissa bits: as exact as an fp32 sum). fp32 inputs: fp32 MFMA
// throughout.
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
    float* seg[2];       // [segment][H][dk][dv]: contributions, then boundary states (0: S, 1: adjoint)
    float* seg_decay;    // [segment][H]
    void* blk[2];        // [block][H][dk][dv] in the input type: S at block starts, adjoint at block ends
};

// tokens per block: fp32 tiles are twice as large, and fp32 MFMA makes the
// quadratic part dearer
template <class T> constexpr int lin_block() { return sizeof(T) == 2 ? 64 : 32; }

// ---------------------------------------------------------------- decays of a block

template <int CTRL> __device__ __forceinline__ float dpp_or_one(float x) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp((int)0x3f800000, (int)__float_as_uint(x), CTRL, 0xF,
                                                                 0xF, false));
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

template <int C, int D> __device__ __forceinline__ void diag_step(float* row, int il, float a, float& acc) {
    if constexpr (D < 16) {
        if constexpr (D == 1) acc *= a; else acc *= dpp_or_one<0x110 + D - 1>(a);   // row_shr: a_{i-D+1}
        if (il >= D) row[il - D] = acc;
        diag_step<C, D + 1>(row, il, a, acc);
    }
}

// One wave, lane = token, `a` its decay (1 past the sequence's end).
template <int C, bool DIAG> __device__ __forceinline__ void block_decays(Decays<C>& s, float a, int lane) {
    float p = a, u = a;
    p *= dpp_or_one<0x111>(p); p *= dpp_or_one<0x112>(p); p *= dpp_or_one<0x114>(p); p *= dpp_or_one<0x118>(p);
    u *= dpp_or_one<0x101>(u); u *= dpp_or_one<0x102>(u); u *= dpp_or_one<0x104>(u); u *= dpp_or_one<0x108>(u);
    const float ux = dpp_or_one<0x101>(u);
    float b[4];
#pragma unroll
    for (int m = 0; m < 4; ++m)
        b[m] = 16 * m < C ? __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(p), 16 * m + 15)) : 1.f;
    const int blk = lane >> 4;
    float pre = 1.f, post = 1.f;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        if (m < blk) pre *= b[m];
        if (m > blk) post *= b[m];
    }
    if (lane < C) {
        s.gam[lane] = pre * p;
        s.suf[lane] = ux * post;
        s.a[lane] = a;
        if constexpr (DIAG) {
            s.row[lane] = p;
            s.col[lane] = ux;
            float* r = s.diag + lane * Decays<C>::DST;
            const int il = lane & 15;
            r[il] = 1.f;
            float acc = 1.f;
            diag_step<C, 1>(r, il, a, acc);
        }
    }
    if (lane == 0) {
        s.total = (b[0] * b[1]) * (b[2] * b[3]);
#pragma unroll
        for (int m = 0; m < 4; ++m) s.blk[m] = b[m];
    }
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

// One segment of one head in one direction: the state's transpose (rows dv,
// columns dk) in accumulators, dk columns split over the waves.
//   !STORE: from zero; writes the segment's contribution and its decay.
//   STORE:  from the boundary state; writes the state before every block.
template <class T, int DK, int DV, int NW, bool STORE>
__global__ void __launch_bounds__(64 * NW) lin_state_kernel(LinParams p) {
    constexpr int C = lin_block<T>(), NT = 64 * NW, NPW = DK / 16 / NW, MT = DV / 16;
    constexpr int SX = tile_stride<T>(DV), SY = tile_stride<T>(DK), PARTS = sizeof(T) == 4 ? 1 : STORE ? 2 : 3;
    using V8 = typename Frag<T>::V;
    extern __shared__ __align__(16) unsigned char smem[];
    lds_poison((uint32_t)(sizeof(Decays<C>) + sizeof(T) * C * (SX + SY)));
    Decays<C>& dec = *reinterpret_cast<Decays<C>*>(smem);
    T* sx = reinterpret_cast<T*>(smem + sizeof(Decays<C>));
    T* sy = sx + C * SX;

    const int tid = threadIdx.x, lane = tid % WAVE, w = tid / WAVE, g = lane >> 4, il = lane & 15;
    const int h = blockIdx.y, rev = blockIdx.z;
    SeqBlock b;
    if (!seq_block(p.map, p.L, blockIdx.x, b)) return;
    const int nc = (b.n + C - 1) / C;
    const size_t at = (size_t)blockIdx.x * p.H + h;
    const T* X = static_cast<const T*>(rev ? p.dO : p.v);
    const T* Y = static_cast<const T*>(rev ? p.q : p.k);
    const size_t rx = (size_t)p.H * DV, ry = (size_t)p.H * DK;

    f32x4 acc[NPW][MT];
#pragma unroll
    for (int x = 0; x < NPW; ++x)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            if constexpr (STORE)
                acc[x][m] = *reinterpret_cast<const f32x4*>(p.seg[rev] + at * (DK * DV) +
                                                            (size_t)(16 * (w * NPW + x) + il) * DV + 16 * m + 4 * g);
            else
                acc[x][m] = zero4();
        }

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
        if constexpr (STORE) {
            T* dst = static_cast<T*>(p.blk[rev]) + ((size_t)((long)blockIdx.x * (p.L / C) + c) * p.H + h) * (DK * DV);
#pragma unroll
            for (int x = 0; x < NPW; ++x)
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    store4(dst + (size_t)(16 * (w * NPW + x) + il) * DV + 16 * m + 4 * g, acc[x][m]);
            if (step == nc - 1) break;
        }
        if (step) __syncthreads();
        stx.store(sx, tid);
        sty.store(sy, tid);
        if (w == 0) block_decays<C, false>(dec, a.value(p, lane), lane);
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
    if constexpr (!STORE) {
#pragma unroll
        for (int x = 0; x < NPW; ++x)
#pragma unroll
            for (int m = 0; m < MT; ++m)
                *reinterpret_cast<f32x4*>(p.seg[rev] + at * (DK * DV) + (size_t)(16 * (w * NPW + x) + il) * DV + 16 * m +
                                          4 * g) = acc[x][m];
        if (tid == 0 && !rev) p.seg_decay[at] = decay;
    }
}

// ---------------------------------------------------------------- scan over segments

// Elementwise over dk x dv, one (sequence, head) per blockIdx.x. Direction 0:
// every segment's contribution is replaced by the state at its start, the end
// is S_T. Direction 1: by the adjoint at its end, the beginning is dS0.
__global__ void __launch_bounds__(256) lin_scan_kernel(LinParams p, int dkdv) {
    lds_poison(0);
    const int s = blockIdx.x / p.H, h = blockIdx.x % p.H, rev = blockIdx.z;
    const int e = 4 * (blockIdx.y * 256 + threadIdx.x);
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
            *reinterpret_cast<f32x4*>(p.seg[rev] + ((size_t)(first + b) * p.H + h) * dkdv + e) = cur;
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
// columns split over the waves; its D tiles are ready A operands of S^T q.
// WHOLE: the segment is the whole sequence, from S0 to S_T.
template <class T, int DK, int DV, int NW, bool WHOLE>
__global__ void __launch_bounds__(64 * NW) lin_out_kernel(LinParams p) {
    constexpr int C = lin_block<T>(), NT = 64 * NW, NPW = DV / 16 / NW, MT = DK / 16, CT = C / 16;
    constexpr int KS = tile_cols<T>(DK) / 32, SK = tile_stride<T>(DK), SV = tile_stride<T>(DV), SP = tile_stride<T>(C);
    constexpr int PARTS = sizeof(T) == 2 && WHOLE ? 3 : 1;
    using V8 = typename Frag<T>::V;
    extern __shared__ __align__(16) unsigned char smem[];
    lds_poison((uint32_t)(sizeof(Decays<C>) + sizeof(T) * C * (2 * SK + SV + SP)));
    Decays<C>& dec = *reinterpret_cast<Decays<C>*>(smem);
    T* sq = reinterpret_cast<T*>(smem + sizeof(Decays<C>));
    T* sk = sq + C * SK;
    T* sv = sk + C * SK;
    T* sp = sv + C * SV;   // [i][j] decayed scores

    const int tid = threadIdx.x, lane = tid % WAVE, w = tid / WAVE, g = lane >> 4, il = lane & 15;
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
    const float* init = WHOLE ? (p.S0 ? p.S0 + ends : nullptr)
                              : p.seg[0] + ((size_t)blockIdx.x * p.H + h) * (DK * DV);
#pragma unroll
    for (int x = 0; x < NPW; ++x)
#pragma unroll
        for (int m = 0; m < MT; ++m) S[x][m] = zero4();
    if (init) {
#pragma unroll
        for (int x = 0; x < NPW; ++x)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    S[x][m][r] = init[(size_t)(16 * m + 4 * g + r) * DV + 16 * (w * NPW + x) + il];
    }
    zero_pad_cols<T, DK>(sq, C, tid, NT);
    zero_pad_cols<T, DK>(sk, C, tid, NT);
    for (int c = 0; c < nc; ++c) {
        if (c) __syncthreads();
        stq.store(sq, tid);
        stk.store(sk, tid);
        stv.store(sv, tid);
        if (w == 0) block_decays<C, true>(dec, a.value(p, lane), lane);
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
                T* out = static_cast<T*>(p.o) + ((size_t)(b.t0 + c * C + 16 * tt + il) * p.H + h) * DV + 4 * g;
#pragma unroll
                for (int x = 0; x < NPW; ++x) store4(out + 16 * (w * NPW + x), acc[x][tt]);
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

// One block of one head. With the start state S and the end adjoint E:
//   dq_i = G_i S dO_i + sum_{j<=i} D_ij (dO_i . v_j) k_j
//   dk_j = d_j E v_j  + sum_{i>=j} D_ij (dO_i . v_j) q_i
//   dv_j = d_j E^T k_j + sum_{i>=j} D_ij (q_i . k_j) dO_i
// and da_t by its definition as a sum over the pairs (j, i), j < t <= i, of
// their products without a_t: M_ij = (q_i . k_j)(dO_i . v_j) weighted with
// a_{j+1}..a_{t-1} and a_{t+1}..a_i, where the start state takes the place of
// an earlier token (r_i = q_i . S dO_i), the end adjoint that of a later one
// (c_j = k_j . E v_j), and both together give <S, E>:
//   R_0[i] = r_i,  R_{t+1}[i] = a_t R_t[i] + M_it        (scan along a row)
//   da_t = sum_{i>=t} a_{t+1}..a_i R_t[i]                (and down a column)
template <class T, int DK, int DV, bool DG> struct LinGradTiles {
    static constexpr int C = lin_block<T>(), NW = (DK > DV ? DK : DV) / 16;
    static constexpr int SK = tile_stride<T>(DK), SV = tile_stride<T>(DV), SP = tile_stride<T>(C), SM = C + 1;
    static constexpr int GROWS = DK < 32 ? 32 : DK;
    Decays<C> dec;
    alignas(16) T q[C * SK], k[C * SK], v[C * SV], dO[C * SV];
    alignas(16) T E[GROWS * SV];
    alignas(16) T p[C * SP], b[C * SP];   // decayed scores and decayed dO . v, [i][j]
    float M[DG ? C * SM : 1];
    float r[DG ? NW * C : 1], c[DG ? NW * C : 1], x[NW];
};

template <class T, int DK, int DV, bool DG>
__global__ void __launch_bounds__(4 * (DK > DV ? DK : DV)) lin_grad_kernel(LinParams p) {
    using L = LinGradTiles<T, DK, DV, DG>;
    constexpr int C = L::C, NW = L::NW, NT = 64 * NW, CT = C / 16, SK = L::SK, SV = L::SV, SP = L::SP, SM = L::SM;
    constexpr int KSK = tile_cols<T>(DK) / 32, KSV = tile_cols<T>(DV) / 32;
    using V8 = typename Frag<T>::V;
    extern __shared__ __align__(16) unsigned char smem[];
    lds_poison((uint32_t)sizeof(L));
    L& s = *reinterpret_cast<L*>(smem);

    const int tid = threadIdx.x, lane = tid % WAVE, w = tid / WAVE, g = lane >> 4, il = lane & 15;
    const int h = blockIdx.y;
    const int per = p.L / C;
    SeqBlock b;
    if (!seq_block(p.map, p.L, blockIdx.x / per, b)) return;
    const int c = blockIdx.x % per;
    const int n = min(C, b.n - c * C);
    if (n <= 0) return;
    const long t0 = b.t0 + (long)c * C;
    const size_t r0 = (size_t)t0 * p.H + h, rk = (size_t)p.H * DK, rv = (size_t)p.H * DV;
    const size_t at = ((size_t)blockIdx.x * p.H + h) * (DK * DV);

    {
        Stage<T, DK, C, NT> a, bb;
        Stage<T, DV, C, NT> cc, dd;
        Stage<T, DV, DK, NT> ee;
        a.load(static_cast<const T*>(p.q) + r0 * DK, rk, n, tid);
        bb.load(static_cast<const T*>(p.k) + r0 * DK, rk, n, tid);
        cc.load(static_cast<const T*>(p.v) + r0 * DV, rv, n, tid);
        dd.load(static_cast<const T*>(p.dO) + r0 * DV, rv, n, tid);
        ee.load(static_cast<const T*>(p.blk[1]) + at, DV, DK, tid);
        if (w == 0) {
            DecayLoad<T> x(p, h);
            x.load(p, t0, h, lane, n);
            block_decays<C, true>(s.dec, x.value(p, lane), lane);
        }
        a.store(s.q, tid);
        bb.store(s.k, tid);
        cc.store(s.v, tid);
        dd.store(s.dO, tid);
        ee.store(s.E, tid);
    }
    zero_pad_cols<T, DK>(s.q, C, tid, NT);
    zero_pad_cols<T, DK>(s.k, C, tid, NT);
    zero_pad_cols<T, DV>(s.v, C, tid, NT);
    zero_pad_cols<T, DV>(s.dO, C, tid, NT);
    zero_pad_cols<T, DV>(s.E, DK, tid, NT);
    if constexpr (DK < 32)   // rows 16..31 of E are contracted over too
        for (int e = tid; e < 16 * SV; e += NT) s.E[16 * SV + e] = T(0);

    // S rows of this wave's dk tile: dv is contracted
    V8 sf[KSV];
    if (w < DK / 16) {
        const T* src = static_cast<const T*>(p.blk[0]) + at + (size_t)(16 * w + il) * DV + 4 * g;
#pragma unroll
        for (int ks = 0; ks < KSV; ++ks) {
            f32x8 x;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                x[m] = from_el(src[32 * ks + m]);
                x[4 + m] = DV >= 32 ? from_el(src[32 * ks + (DV >= 32 ? 16 : 0) + m]) : 0.f;
            }
            sf[ks] = narrow<T>(x);
        }
    }
    __syncthreads();

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
        if constexpr (DG) {
            float* m = s.M + (16 * ti + il) * SM + 16 * tj + 4 * g;
#pragma unroll
            for (int r = 0; r < 4; ++r) m[r] = x[r] * y[r];
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const bool in = tj < ti || 4 * g + r <= il;
            x[r] = in ? x[r] * d[r] : 0.f;
            y[r] = in ? y[r] * d[r] : 0.f;
        }
        const int to = (16 * ti + il) * SP + 16 * tj + 4 * g;
        store4(s.p + to, x);
        store4(s.b + to, y);
        if (ti == tj && ti % 2 == 0) {   // the other half of a 32-deep step
            store4(s.p + to + 16, zero4());
            store4(s.b + to + 16, zero4());
        }
    }

    // products with the boundary states
    f32x4 aq[CT], ak[CT], av[CT];
#pragma unroll
    for (int tt = 0; tt < CT; ++tt) aq[tt] = ak[tt] = av[tt] = zero4();
    if (w < DK / 16) {
        float xe = 0.f;
#pragma unroll
        for (int ks = 0; ks < KSV; ++ks) {
            const V8 ef = frag_kpos(s.E, SV, 16 * w + il, 32 * ks, g);
            if constexpr (DG) {
                const f32x8 e8 = widen(ef) * widen(sf[ks]);
                xe += ((e8[0] + e8[1]) + (e8[2] + e8[3])) + ((e8[4] + e8[5]) + (e8[6] + e8[7]));
            }
#pragma unroll
            for (int tt = 0; tt < CT; ++tt) {
                aq[tt] = mma(sf[ks], frag_kpos(s.dO, SV, 16 * tt + il, 32 * ks, g), aq[tt]);
                ak[tt] = mma(ef, frag_kpos(s.v, SV, 16 * tt + il, 32 * ks, g), ak[tt]);
            }
        }
        if constexpr (DG) {
            xe = wave_sum(xe);
            if (lane == 0) s.x[w] = xe;
#pragma unroll
            for (int tt = 0; tt < CT; ++tt) {
                const int i = 16 * tt + il;
                float rr = 0.f, cc = 0.f;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    rr += aq[tt][r] * from_el(s.q[i * SK + 16 * w + 4 * g + r]);
                    cc += ak[tt][r] * from_el(s.k[i * SK + 16 * w + 4 * g + r]);
                }
                rr += __shfl_xor(rr, 16, WAVE);
                rr += __shfl_xor(rr, 32, WAVE);
                cc += __shfl_xor(cc, 16, WAVE);
                cc += __shfl_xor(cc, 32, WAVE);
                if (g == 0) {
                    s.r[w * C + i] = rr;
                    s.c[w * C + i] = cc;
                }
            }
        }
    }
    if (w < DV / 16) {
#pragma unroll
        for (int ks = 0; ks < KSK; ++ks) {
            const V8 ef = frag_tr(s.E, SV, 32 * ks, 16 * w, g, il);
#pragma unroll
            for (int tt = 0; tt < CT; ++tt) av[tt] = mma(ef, frag_kpos(s.k, SK, 16 * tt + il, 32 * ks, g), av[tt]);
        }
    }
#pragma unroll
    for (int tt = 0; tt < CT; ++tt) {
        const float gi = s.dec.gam[16 * tt + il], di = s.dec.suf[16 * tt + il];
        aq[tt] *= gi;
        ak[tt] *= di;
        av[tt] *= di;
    }
    __syncthreads();

    // products inside the block
    constexpr int KC = C / 32;
    if (w < DK / 16) {
        V8 kf[KC], qf[KC];
#pragma unroll
        for (int ks = 0; ks < KC; ++ks) {
            kf[ks] = frag_tr(s.k, SK, 32 * ks, 16 * w, g, il);
            qf[ks] = frag_tr(s.q, SK, 32 * ks, 16 * w, g, il);
        }
#pragma unroll
        for (int tt = 0; tt < CT; ++tt) {
#pragma unroll
            for (int ks = 0; ks <= tt / 2; ++ks) aq[tt] = mma(kf[ks], frag_kpos(s.b, SP, 16 * tt + il, 32 * ks, g), aq[tt]);
#pragma unroll
            for (int ks = tt / 2; ks < KC; ++ks)
                ak[tt] = mma(qf[ks], frag_tr(s.b, SP, 32 * ks, 16 * tt, g, il), ak[tt]);
            const int i = 16 * tt + il;
            if (i < n) {
                const size_t to = (r0 + (size_t)i * p.H) * DK + 16 * w + 4 * g;
                store4(static_cast<T*>(p.dq) + to, aq[tt]);
                store4(static_cast<T*>(p.dk) + to, ak[tt]);
            }
        }
    }
    if (w < DV / 16) {
        V8 of[KC];
#pragma unroll
        for (int ks = 0; ks < KC; ++ks) of[ks] = frag_tr(s.dO, SV, 32 * ks, 16 * w, g, il);
#pragma unroll
        for (int tt = 0; tt < CT; ++tt) {
#pragma unroll
            for (int ks = tt / 2; ks < KC; ++ks)
                av[tt] = mma(of[ks], frag_tr(s.p, SP, 32 * ks, 16 * tt, g, il), av[tt]);
            const int i = 16 * tt + il;
            if (i < n) store4(static_cast<T*>(p.dv) + (r0 + (size_t)i * p.H) * DV + 16 * w + 4 * g, av[tt]);
        }
    }

    if constexpr (DG) {
        if (w == 0) {
            const int i = lane % C;   // C = 32: the upper lanes repeat the lower ones
            constexpr int NK = DK / 16;
            float R = 0.f, cl = 0.f, X = 0.f, RC = 0.f;
            for (int m = 0; m < NK; ++m) {
                R += s.r[m * C + i];
                cl += s.c[m * C + i];
                X += s.x[m];
            }
            // along the rows, in place: M_it becomes R_t[i]; the row of the end
            // adjoint (M_it = c_t, R_0 = <S, E>) is kept by lane t
            float* row = s.M + i * SM;
            for (int t = 0; t < C; ++t) {
                const float m = row[t], at = s.dec.a[t];
                row[t] = R;
                if (t == i) RC = X;
                R = at * R + (t < i ? m : 0.f);
                X = at * X + __shfl(cl, t, WAVE);
            }
            __builtin_amdgcn_wave_barrier();
            // down the columns
            float acc = RC;
            for (int j = C - 1; j >= 0; --j) {
                if (j >= i) acc = s.M[j * SM + i] + (j == C - 1 ? acc : s.dec.a[j + 1] * acc);
            }
            if (lane < n) store1(static_cast<T*>(p.dgate) + (size_t)(t0 + lane) * p.H + h, acc);
        }
    }
}

// ---------------------------------------------------------------- decode

// S' = a S + k v^T, o = S'^T q = a (S^T q) + (k . q) v, the state streamed once
// in and once out. One workgroup takes DVW of a head's dv columns; a column
// needs no other, so few heads spread over more workgroups.
template <class T, int DK, int DVW, int NT>
__global__ void __launch_bounds__(NT) lin_decode_kernel(const T* __restrict__ q, const T* __restrict__ k,
                                                        const T* __restrict__ v, const void* __restrict__ gate,
                                                        float* __restrict__ S, T* __restrict__ o, int H, int DV,
                                                        int head_gate) {
    constexpr int CG = DVW / 4, RG = NT / CG, RPT = DK / RG, NW = NT / WAVE;
    static_assert(NT % WAVE == 0 && DK % RG == 0 && RPT >= 1, "decode tiling");
    lds_poison(0);
    __shared__ float s_k[DK], s_q[DK], s_v[DVW], s_red[NW][DVW], s_kq[NW];
    const size_t pair = blockIdx.x;
    const int c0 = blockIdx.y * DVW, t = threadIdx.x, cg = t % CG, rg = t / CG, lane = t % WAVE, w = t / WAVE;
    float kq = 0.f;
    for (int e = t; e < DK; e += NT) {
        const float kv = ld_in(k + pair * DK + e), qv = ld_in(q + pair * DK + e);
        s_k[e] = kv;
        s_q[e] = qv;
        kq += kv * qv;
    }
    for (int e = t; e < DVW; e += NT) s_v[e] = ld_in(v + pair * DV + c0 + e);
    const float a = head_gate ? static_cast<const float*>(gate)[pair % H] : ld_in(static_cast<const T*>(gate) + pair);
    f32x4* Sp = reinterpret_cast<f32x4*>(S + pair * DK * DV + c0);
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
    if (t < DVW) {
        float acc = 0.f, dot = 0.f;
#pragma unroll
        for (int m = 0; m < NW; ++m) {
            acc += s_red[m][t];
            dot += s_kq[m];
        }
        store1(o + pair * DV + c0 + t, a * acc + dot * s_v[t]);
    }
}

size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

// Tokens per segment. Enough segments that every CU has two workgroups, at
// least 128 tokens each so that the extra read of k and v and the states are
// paid for, and one segment per sequence where sequences are short.
int segment_tokens(int T, int N, int H, bool packed) {
    const long tokens = packed ? T : (long)T * N;
    const long want = tokens * H / 512;
    long L = (want + 63) / 64 * 64;
    if (L < 128) L = 128;
    const long whole = ((long)T + 63) / 64 * 64;
    return (int)(L < whole ? L : (whole > 0 ? whole : 64));
}
bool whole_sequences(int T) { return T <= 256; }

struct LinWorkspace {
    size_t seg[2], decay, blk[2], total;
};
LinWorkspace workspace_layout(int T, int N, int H, int dk, int dv, bool packed, bool bf16, bool grad, int L) {
    const size_t segs = (size_t)seq_blocks_bound(T, N, L, packed) * H, state = (size_t)dk * dv;
    const size_t blocks = segs * (L / (bf16 ? 64 : 32));
    LinWorkspace w{};
    size_t at = 0;
    auto take = [&](size_t bytes) { const size_t r = at; at += al256(bytes); return r; };
    w.seg[0] = take(segs * state * 4);
    w.decay = take(segs * 4);
    if (grad) {
        w.seg[1] = take(segs * state * 4);
        w.blk[0] = take(blocks * state * (bf16 ? 2 : 4));
        w.blk[1] = take(blocks * state * (bf16 ? 2 : 4));
    }
    w.total = at;
    return w;
}

template <class K> hipError_t launch(K kern, dim3 grid, int threads, size_t lds, hipStream_t stream, const LinParams& p) {
    if (lds > 65536) {
        const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kern, grid, dim3(threads), lds, stream, p);
    return hipGetLastError();
}

template <class T, int DK, int DV, bool STORE>
hipError_t launch_state(const LinParams& p, int segs, int dirs, hipStream_t st) {
    constexpr int NW = DK / 16 < 4 ? DK / 16 : 4, C = lin_block<T>();
    return launch(lin_state_kernel<T, DK, DV, NW, STORE>, dim3(segs, p.H, dirs), 64 * NW,
                  sizeof(Decays<C>) + sizeof(T) * C * (tile_stride<T>(DK) + tile_stride<T>(DV)), st, p);
}

template <class T, int DK, int DV, bool WHOLE> hipError_t launch_out(const LinParams& p, int segs, hipStream_t st) {
    constexpr int NW = DV / 16 < 4 ? DV / 16 : 4, C = lin_block<T>();
    return launch(lin_out_kernel<T, DK, DV, NW, WHOLE>, dim3(segs, p.H), 64 * NW,
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
    hipLaunchKernelGGL(lin_scan_kernel, dim3(p.map.N * p.H, (DK * DV / 4 + 255) / 256, 1), dim3(256), 0, a.stream, p, DK * DV);
    e = hipGetLastError();
    if (e != hipSuccess || p.map.T == 0) return e;
    return launch_out<T, DK, DV, false>(p, segs, a.stream);
}

template <class T, int DK, int DV> hipError_t backward(const LinParams& p, const LinArgs& a) {
    const bool packed = p.map.cu != nullptr;
    const int segs = (int)seq_blocks_bound(p.map.T, p.map.N, p.L, packed);
    hipError_t e = hipSuccess;
    if (p.map.T > 0) e = launch_state<T, DK, DV, false>(p, segs, 2, a.stream);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(lin_scan_kernel, dim3(p.map.N * p.H, (DK * DV / 4 + 255) / 256, 2), dim3(256), 0, a.stream, p, DK * DV);
    e = hipGetLastError();
    if (e != hipSuccess || p.map.T == 0) return e;
    e = launch_state<T, DK, DV, true>(p, segs, 2, a.stream);
    if (e != hipSuccess) return e;
    const dim3 grid(segs * (p.L / lin_block<T>()), p.H);
    constexpr int NT = 4 * (DK > DV ? DK : DV);
    if (p.head_gate) return launch(lin_grad_kernel<T, DK, DV, false>, grid, NT, sizeof(LinGradTiles<T, DK, DV, false>), a.stream, p);
    return launch(lin_grad_kernel<T, DK, DV, true>, grid, NT, sizeof(LinGradTiles<T, DK, DV, true>), a.stream, p);
}

template <class T, int DK, int DV> hipError_t decode(const LinDecodeArgs& a) {
    const int pairs = a.N * a.H;
    auto go = [&](auto kern, int threads, int cols) {
        hipLaunchKernelGGL(kern, dim3(pairs, DV / cols), dim3(threads), 0, a.stream, (const T*)a.q, (const T*)a.k,
                           (const T*)a.v, a.gate, a.S, (T*)a.o, a.H, DV, (int)a.head_gate);
        return hipGetLastError();
    };
    constexpr int NT = DK * DV / 4 < 512 ? DK * DV / 4 : 512;
    // under two heads per CU the columns of a head are split over workgroups
    if constexpr (DV > 32 && DK >= 32)
        if (pairs < 512) return go(lin_decode_kernel<T, DK, 32, (DK * 8 < 512 ? DK * 8 : 512)>, DK * 8 < 512 ? DK * 8 : 512, 32);
    return go(lin_decode_kernel<T, DK, DV, NT>, NT, DV);
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
    p.L = segment_tokens(a.T, a.N, a.H, packed);
    const LinWorkspace w = workspace_layout(a.T, a.N, a.H, a.dk, a.dv, packed, a.bf16, grad, p.L);
    char* base = static_cast<char*>(a.workspace);
    for (int d = 0; d < 2; ++d) {
        p.seg[d] = reinterpret_cast<float*>(base + w.seg[d]);
        p.blk[d] = base + w.blk[d];
    }
    p.seg_decay = reinterpret_cast<float*>(base + w.decay);
    return p;
}

}  // namespace

size_t lin_workspace_bytes(int B, int H, int T, int dk, int dv, bool packed, int N, bool bf16, bool grad) {
    if (!packed) N = B;
    if (!grad && T > 0 && whole_sequences(T)) return 256;
    const size_t n = workspace_layout(T, N, H, dk, dv, packed, bf16, grad, segment_tokens(T, N, H, packed)).total;
    return n ? n : 256;
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
