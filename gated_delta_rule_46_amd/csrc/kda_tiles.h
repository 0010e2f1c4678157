// LDS tiles and their MFMA fragments, shared by the linear-attention and the
// window-attention kernels (gfx950).
//
// A tile holds rows (tokens) x D columns of the input type, row-major. Its
// row stride is padded so that the reads below spread over the LDS banks:
//   nat   one row per lane, 8 values along it     (contraction over columns)
//   kpos  the same in the kpos order of kda_common.h, for products whose
//         other operand comes straight from accumulator registers
//   tr    one column per lane, 8 rows in the kpos order (contraction over
//         rows): bf16 by the transposing LDS read, fp32 by scalar reads
// Every contraction step is 32 deep; a tile of 16 columns is padded to 32
// with zero columns.
#pragma once

#include "kda_common.h"

namespace kda {

template <class T> struct Frag;
template <> struct Frag<uint16_t> { using V = bf16x8; };
template <> struct Frag<float> { using V = f32x8; };

typedef short s16x4 __attribute__((ext_vector_type(4)));

// row stride in elements: four dwords past a multiple of 32, the banks. Eight
// consecutive rows are then 4 banks apart and cover all of them with the 16
// bytes of a nat read each, or with a lane group's 8 dwords of a tr read twice;
// so are 16 rows with the 8 bytes that two lane groups of a kpos read take. No
// read above conflicts (with eight dwords, nat and kpos take twice the cycles).
template <class T> __host__ __device__ constexpr int tile_cols(int d) { return d < 32 ? 32 : d; }
template <class T> __host__ __device__ constexpr int tile_stride(int d) {
    return tile_cols<T>(d) + (sizeof(T) == 2 ? 8 : 4);
}

__device__ __forceinline__ bf16x8 frag_nat(const uint16_t* t, int st, int row, int k0, int g) {
    return *reinterpret_cast<const bf16x8*>(t + row * st + k0 + 8 * g);
}
__device__ __forceinline__ f32x8 frag_nat(const float* t, int st, int row, int k0, int g) {
    const f32x4* p = reinterpret_cast<const f32x4*>(t + row * st + k0 + 8 * g);
    const f32x4 a = p[0], b = p[1];
    return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

__device__ __forceinline__ bf16x8 frag_kpos(const uint16_t* t, int st, int row, int k0, int g) {
    const uint2 a = *reinterpret_cast<const uint2*>(t + row * st + k0 + 4 * g);
    const uint2 b = *reinterpret_cast<const uint2*>(t + row * st + k0 + 16 + 4 * g);
    const uint4 u = make_uint4(a.x, a.y, b.x, b.y);
    return __builtin_bit_cast(bf16x8, u);
}
__device__ __forceinline__ f32x8 frag_kpos(const float* t, int st, int row, int k0, int g) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(t + row * st + k0 + 4 * g);
    const f32x4 b = *reinterpret_cast<const f32x4*>(t + row * st + k0 + 16 + 4 * g);
    return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// column c0 + i (i = lane % 16), rows r0 + kpos(g, 0..7)
__device__ __forceinline__ bf16x8 frag_tr(const uint16_t* t, int st, int r0, int c0, int g, int i) {
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const uint16_t* p = t + (r0 + 4 * g + (i >> 2)) * st + c0 + 4 * (i & 3);
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 16 * st));
    const auto u = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8, u);
}
__device__ __forceinline__ f32x8 frag_tr(const float* t, int st, int r0, int c0, int g, int i) {
    f32x8 r;
    const float* p = t + (r0 + 4 * g) * st + c0 + i;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        r[m] = p[m * st];
        r[4 + m] = p[(16 + m) * st];
    }
    return r;
}

__device__ __forceinline__ f32x8 widen(const bf16x8& x) { return __builtin_convertvector(x, f32x8); }
__device__ __forceinline__ f32x8 widen(const f32x8& x) { return x; }

// fp32 values as an operand of the input type (bf16: rounded to nearest)
template <class T> __device__ __forceinline__ typename Frag<T>::V narrow(const f32x8& x);
template <> __device__ __forceinline__ bf16x8 narrow<uint16_t>(const f32x8& x) { return __builtin_convertvector(x, bf16x8); }
template <> __device__ __forceinline__ f32x8 narrow<float>(const f32x8& x) { return x; }

// four values to consecutive elements (8 or 16 bytes, aligned)
__device__ __forceinline__ void store4(uint16_t* p, const f32x4& x) {
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<bf16x4*>(p) = __builtin_convertvector(x, bf16x4);
}
__device__ __forceinline__ void store4(float* p, const f32x4& x) { *reinterpret_cast<f32x4*>(p) = x; }

// Columns 4 g + (0..3) of two neighbouring 16-column tiles of a row: the lane groups
// swap halves, so that bf16 goes out 16 bytes a lane, 64 in a row, instead of 8 and 32.
__device__ __forceinline__ void store_pair(uint16_t* row, const f32x4& x, const f32x4& y, int g) {
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    typedef uint32_t u2 __attribute__((ext_vector_type(2)));
    const u2 a = __builtin_bit_cast(u2, __builtin_convertvector(x, bf16x4));
    const u2 b = __builtin_bit_cast(u2, __builtin_convertvector(y, bf16x4));
    // odd groups of the first operand against even ones of the second
    const auto s0 = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto s1 = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    *reinterpret_cast<uint4*>(row + 16 * (g & 1) + 8 * (g >> 1)) = make_uint4(s0[0], s1[0], s0[1], s1[1]);
}
__device__ __forceinline__ void store_pair(float* row, const f32x4& x, const f32x4& y, int g) {
    *reinterpret_cast<f32x4*>(row + 4 * g) = x;
    *reinterpret_cast<f32x4*>(row + 16 + 4 * g) = y;
}

// four elements as they lie in memory, held whole (arrays of 16-bit elements
// would take a register each), and their values
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <class T> struct Raw4;
template <> struct Raw4<uint16_t> { using V = u32x2; };
template <> struct Raw4<float> { using V = u32x4; };
__device__ __forceinline__ f32x4 values(const u32x2& x) {
    return f32x4{__uint_as_float(x[0] << 16), __uint_as_float(x[0] & 0xffff0000u), __uint_as_float(x[1] << 16),
                 __uint_as_float(x[1] & 0xffff0000u)};
}
__device__ __forceinline__ f32x4 values(const u32x4& x) { return __builtin_bit_cast(f32x4, x); }
__device__ __forceinline__ float from_el(uint16_t x) { return bf16_bits_to_f32(x); }
__device__ __forceinline__ float from_el(float x) { return x; }
__device__ __forceinline__ void store1(uint16_t* p, float x) {
    *p = __builtin_bit_cast(uint16_t, (__bf16)x);
}
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }

// A tile on its way from global memory to LDS through registers, 16 bytes a
// thread and step: rows row0 + (0..R-1) of `stride` elements. The loads go
// through a buffer descriptor that ends behind row `valid` - 1, so that later
// rows read as zeros and touch no memory, with no branch around a load.
template <class T, int D, int R, int NT> struct Stage {
    static constexpr int PER = 16 / (int)sizeof(T), CPR = D / PER, TOT = R * CPR, N = (TOT + NT - 1) / NT;
    u32x4 r[N];
    __device__ __forceinline__ void load(const T* base, size_t stride, int valid, int tid) {
        const uint32_t bytes = (uint32_t)stride * (uint32_t)sizeof(T);
        // said to be the same in every lane: a clamp is vector arithmetic, and a
        // descriptor in vector registers costs a loop around each load
        const uint32_t size = __builtin_amdgcn_readfirstlane(min(max(valid, 0), R) * (int)bytes);
        const auto rsrc = make_rsrc(base, size);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int e = tid + n * NT;
            if (TOT % NT == 0 || e < TOT)
                r[n] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, (uint32_t)(e / CPR) * bytes + (uint32_t)(e % CPR) * 16u, 0, 0);
        }
    }
    __device__ __forceinline__ void store(T* tile, int tid) const {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int e = tid + n * NT;
            if (TOT % NT == 0 || e < TOT) *reinterpret_cast<u32x4*>(tile + (e / CPR) * tile_stride<T>(D) + (e % CPR) * PER) = r[n];
        }
    }
};

// number of the wave in its workgroup, as a scalar: branches and addresses that
// depend on it stay out of the vector registers
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE); }

// The same value, unknown to the compiler from here on: LDS addresses formed from
// it inside a loop stay there, where a few additions cost less than the hundreds
// of registers that hoisting every one of them out of the loop takes (and spills).
__device__ __forceinline__ int here(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

// The same for values held over a loop as they lie in memory, so that what is
// unpacked from them is not hoisted and held instead.
template <class V> __device__ __forceinline__ V raw_here(V x) {
    asm volatile("" : "+v"(x));
    return x;
}
// zero columns D..31 of a narrow tile
template <class T, int D> __device__ __forceinline__ void zero_pad_cols(T* tile, int rows, int tid, int nt) {
    if constexpr (D < 32) {
        for (int e = tid; e < rows * (32 - D); e += nt) tile[(e / (32 - D)) * tile_stride<T>(D) + D + e % (32 - D)] = T(0);
    }
}

// ---------------------------------------------------------------- sequences
// Blocks of L tokens over every sequence. Fixed length: block v is block
// v % nb of sequence v / nb. Packed (cu): sequence s owns the block numbers
// from cu[s] / L + s up to cu[s+1] / L + s + 1, which is at least
// ceil(length / L) numbers and needs no index built beforehand; numbers past
// a sequence's last block are empty. Offsets are clamped to [0, T], so that
// rows behind the last sequence are never touched.
struct SeqMap {
    const int32_t* cu;   // null: fixed length
    int T, N;
};
struct SeqBlock {
    int seq, idx;    // sequence, block within it
    long t0;         // first token, flattened over the batch
    int n;           // tokens in the block
    int len;         // tokens of the sequence
    int first;       // number of the sequence's first block
};
__host__ __device__ inline long seq_blocks_bound(int T, int N, int L, bool packed) {
    return packed ? (long)(T / L) + N + 1 : (long)N * ((T + L - 1) / L);
}
__device__ __forceinline__ int seq_offset(const SeqMap& m, int s) { return min(max(m.cu[s], 0), m.T); }
__device__ __forceinline__ bool seq_block(const SeqMap& m, int L, int v, SeqBlock& b) {
    if (m.cu == nullptr) {
        const int nb = (m.T + L - 1) / L;
        b.seq = v / nb;
        b.idx = v % nb;
        b.first = b.seq * nb;
        b.len = m.T;
        b.t0 = (long)b.seq * m.T + (long)b.idx * L;
    } else {
        int lo = 0, hi = m.N - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (seq_offset(m, mid) / L + mid <= v) lo = mid; else hi = mid - 1;
        }
        const int c0 = seq_offset(m, lo);
        b.seq = lo;
        b.first = c0 / L + lo;
        b.idx = v - b.first;
        b.len = max(seq_offset(m, lo + 1) - c0, 0);
        b.t0 = (long)c0 + (long)b.idx * L;
    }
    b.n = b.idx < 0 ? 0 : min(L, b.len - b.idx * L);
    return b.n > 0;
}

// Runs `f` with the constant D for a head size d.
#define KDA_SWITCH_DIM(d, D, ...)                                      \
    [&] {                                                              \
        switch (d) {                                                   \
            case 16: { constexpr int D = 16; return __VA_ARGS__(); }   \
            case 32: { constexpr int D = 32; return __VA_ARGS__(); }   \
            case 64: { constexpr int D = 64; return __VA_ARGS__(); }   \
            default: { constexpr int D = 128; return __VA_ARGS__(); }  \
        }                                                              \
    }()

}  // namespace kda
