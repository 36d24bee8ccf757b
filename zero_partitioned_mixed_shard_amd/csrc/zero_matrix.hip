// zero_matrix.hip -- steps of whole matrices: orthogonalisation by Newton-Schulz
// products (zero_orthogonalize) and the Muon step of an owner's matrices
// (zero_muon_step), over a plan of matrices of any sizes.
//
// Mathematics.  X is the matrix in its wide form (m <= n; a tall matrix is
// transposed on the way in and out), divided by its Frobenius norm; then `steps`
// times
//     A = X X^T,   B = b A + c A A,   X <- a X + B X,
// which applies the polynomial a x + b x^3 + c x^5 to the singular values and
// leaves the singular vectors.  A and A A are symmetric: only the tiles on and
// below the diagonal are computed, and written twice.  Per step that is
// 3 m^2 n + m^3 operations where products that know nothing of the symmetry take
// 4 m^2 n + 2 m^3.
//
// Numerics.  The products run on the matrix cores in fp16 with fp32 sums.  fp16 has
// three bits more than bf16 at the same rate, and its range is enough here: a
// matrix's entries are bounded by its largest singular value, which the host bounds
// for the given coefficients (at most 1.75), so X is kept times 2^15 and A times
// 2^14 and nothing overflows, while entries down to 2^-29 stay normal.  X is kept in
// two parts, hi = fp16(x) and lo = fp16(x - hi).  The products read hi alone; the
// linear term a X takes both.  A direction of small singular values is multiplied by
// a in every step (485 times in 5 steps), and so would be the rounding of X; the two
// parts keep that term to 22 bits.  Relative error of the result (2-norm), against 64
// bits, of 512 x 1376: a normal matrix 1.4e-3 without lo and 1.6e-3 with it (the
// rounding of B, the same either way), one of rank 32 with 5 % of noise 6e-3 and
// 2e-4, one of rank 1 with 0.1 % of noise 0.12 and 2e-4; in bf16 0.011, 0.05 and 1.
// With `precise` A and B have two parts too and every product is hi hi + hi lo +
// lo hi, three times the matrix work, for results in 32 bits.

#include <math.h>
#include <string.h>

#include <algorithm>
#include <new>
#include <vector>

#include "zero_common.h"

namespace {

typedef _Float16 f16;
typedef f16 f16x4 __attribute__((ext_vector_type(4)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef __fp16 fp16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) fp16x4 lds_fp16x4;

// Powers of two that X, A and B are kept times (B's goes by its bound, on the host).
constexpr float kScaleX = 32768.0f, kScaleA = 16384.0f;
// Bound of the singular values in all steps: kScaleX * 1.75 and kScaleA * 1.75^2 are
// below fp16's 65504.
constexpr double kMostSigma = 1.75;
constexpr int64_t kMostLong = 4194240, kMostShort = 65536;   // sides of a matrix
constexpr int kBK = 64;                    // depth of a K step: 128 bytes of a row
constexpr int kUnitM = 64, kUnitN = 128;   // elements of a unit of the streaming passes

// A matrix of the plan, as the kernels read it.
struct Mat {
    const void* src;            // orthogonalize: the matrix and its result
    void* dst;
    int64_t offset;             // muon: its first element in the shard
    int64_t src_ld, dst_ld;     // elements between rows
    int64_t x[2], a, b;         // byte offsets of its planes in the workspace
    int64_t plane_x, plane_a;   // bytes of a plane of X, and of A or B
    int64_t part0;              // its first partial of the norm
    int32_t rows, cols;
    int32_t m, n, mp, np;       // its wide form, and that padded to whole tiles
    int32_t tall;               // rows > cols
    int32_t src_dtype, dst_dtype;
    int32_t n_parts, pad0, pad1;
};
// A tile or unit: which matrix, and where.
struct Item {
    uint32_t mat;
    uint16_t i, j;
};
// Matrices that go through the steps together.
struct Group {
    int64_t mat0, n_mats, unit0, n_units, tri0, n_tri, full0, n_full;
    int64_t inv_off, part_off;  // the norms' factors and partials in the workspace
    int32_t tile, pad;
};
struct Head {
    uint64_t magic;
    int64_t n_groups, groups_off, mats_off, items_off, bytes;
};
constexpr uint64_t kMagic = 0x7a65726f6d617431ull;

// What a call passes to every kernel.
struct Step {
    const Mat* mats;
    const Item* items;      // of the launch
    int64_t n_items;
    char* ws;
    const zero_step_result* res;   // NULL: orthogonalize
    int64_t inv_off, part_off;
};
struct NsConsts {
    float a, b, c, eps;
    float scale_b;          // B is kept times this
};
struct MuonConsts {
    float momentum, decay, lr, max_norm;
    int32_t nesterov, scaling;
};
struct MuonBufs {
    float* master;
    float* momentum;
    uint16_t* p16;
    const uint16_t* g16;
};

__device__ __forceinline__ bool skipped(const zero_step_result* res) {
    return res != nullptr && res->overflow != 0;
}

// Unit of block b of n, so that consecutive units go to one XCD (workgroups are dealt
// to the 8 XCDs in turn) in groups of G; the blocks past the last whole group keep
// their own.
template <int G>
__device__ __forceinline__ int64_t item_of(int64_t b, int64_t n) {
    constexpr int64_t group = 8 * G;
    const int64_t a = b & ~(group - 1);
    if (a + group > n) return b;
    const int64_t r = b - a;
    return a + (r & 7) * G + (r >> 3);
}

// ------------------------------------------------------------ 16 bits ------
__device__ __forceinline__ float widen16(int dt, uint16_t b) {
    return dt == ZERO_FP16 ? (float)__builtin_bit_cast(f16, b) : __uint_as_float((uint32_t)b << 16);
}
// Nearest, ties to even; overflow gives inf, NaN stays (quiet) NaN.
__device__ __forceinline__ uint16_t narrow16(int dt, float f) {
    if (dt == ZERO_FP16) return __builtin_bit_cast(uint16_t, (f16)f);
    const uint32_t u = __float_as_uint(f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((u >> 16) | 0x0040u);
    return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}
__device__ __forceinline__ float load_elem(const void* p, int64_t e, int dt) {
    return dt == ZERO_FP32 ? ((const float*)p)[e] : widen16(dt, ((const uint16_t*)p)[e]);
}

// ------------------------------------------------------------ norm, init ----
// The element of the update at (row, col) of a matrix.  Source of the two
// streaming passes: orthogonalize reads the matrix, the Muon step makes the update of
// gradient and momentum (and stores the momentum in the first pass; the second makes
// the same value again from what was stored).
struct OrthSource {
    __device__ void begin(const Step&) {}
    template <bool FIRST>
    __device__ __forceinline__ float get(const Mat& t, int64_t row, int64_t col) const {
        return load_elem(t.src, row * t.src_ld + col, t.src_dtype);
    }
};
template <int DT>
struct MuonSource {
    MuonBufs p;
    MuonConsts c;
    float inv, coef;
    __device__ void begin(const Step& s) {
        inv = s.res->inv_scale;
        coef = 1.0f;
        if (c.max_norm > 0.0f) {
            const double q = (double)c.max_norm / (sqrt(s.res->sumsq) + 1e-6);
            if (q < 1.0) coef = (float)q;
        }
    }
    template <bool FIRST>
    __device__ __forceinline__ float get(const Mat& t, int64_t row, int64_t col) const {
        const int64_t e = t.offset + row * t.cols + col;
        const float g = widen16(DT, p.g16[e]) * inv * coef;
        float mo = p.momentum[e];
        if (FIRST) {
            mo = c.momentum * mo + g;
            p.momentum[e] = mo;
        }
        return c.nesterov ? g + c.momentum * mo : mo;
    }
};

// First pass: the sum of squares of every unit's elements, in fp64.
template <typename Source>
__global__ void __launch_bounds__(kThreads)
matrix_norm_kernel(Step s, Source src) {
    if (skipped(s.res)) return;
    src.begin(s);
    const int64_t idx = item_of<8>(blockIdx.x, s.n_items);
    const Item it = s.items[idx];
    const Mat t = s.mats[it.mat];
    // the unit's rows and columns in the matrix as it lies in memory
    const int64_t r0 = (int64_t)(t.tall ? it.j * kUnitN : it.i * kUnitM);
    const int64_t c0 = (int64_t)(t.tall ? it.i * kUnitM : it.j * kUnitN);
    const int nr = t.tall ? kUnitN : kUnitM, lc = t.tall ? 6 : 7;
    double sum = 0.0;
    for (int e = threadIdx.x; e < (nr << lc); e += kThreads) {
        const int64_t row = r0 + (e >> lc), col = c0 + (e & ((1 << lc) - 1));
        if (row < t.rows && col < t.cols) {
            const double v = (double)src.template get<true>(t, row, col);
            sum = fma(v, v, sum);
        }
    }
    __shared__ double part[kThreads / 64];
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0)
        ((double*)(s.ws + s.part_off))[idx] = (part[0] + part[1]) + (part[2] + part[3]);
}

// One block per matrix: its factor kScaleX / (norm + eps), the partials in order.
__global__ void __launch_bounds__(kThreads)
matrix_factor_kernel(Step s, float eps) {
    if (skipped(s.res)) return;
    const Mat t = s.mats[blockIdx.x];
    const double* p = (const double*)(s.ws + s.part_off) + t.part0;
    double sum = 0.0;
    for (int k = threadIdx.x; k < t.n_parts; k += kThreads) sum += p[k];
    __shared__ double part[kThreads / 64];
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        const double norm = sqrt((part[0] + part[1]) + (part[2] + part[3]));
        ((float*)(s.ws + s.inv_off))[blockIdx.x] = (float)((double)kScaleX / (norm + (double)eps));
    }
}

__device__ __forceinline__ void split(float v, f16& hi, f16& lo) {
    hi = (f16)v;
    lo = (f16)(v - (float)hi);
}

// Second pass: X in its wide form, both parts, zero in the padding.
template <typename Source>
__global__ void __launch_bounds__(kThreads)
matrix_init_kernel(Step s, int64_t mat0, Source src) {
    if (skipped(s.res)) return;
    src.begin(s);
    __shared__ float turn[kUnitN * (kUnitM + 1)];
    const Item it = s.items[item_of<8>(blockIdx.x, s.n_items)];
    const Mat t = s.mats[it.mat];
    const float inv = ((const float*)(s.ws + s.inv_off))[it.mat - mat0];
    const int i0 = it.i * kUnitM, j0 = it.j * kUnitN;
    if (t.tall) {
        for (int e = threadIdx.x; e < kUnitM * kUnitN; e += kThreads) {
            const int r = e >> 6, c = e & 63;
            const int64_t row = j0 + r, col = i0 + c;
            turn[r * (kUnitM + 1) + c] =
                row < t.rows && col < t.cols ? src.template get<false>(t, row, col) : 0.0f;
        }
        __syncthreads();
    }
    f16* x = (f16*)(s.ws + t.x[0]);
    f16* y = (f16*)(s.ws + t.x[0] + t.plane_x);
    for (int e = threadIdx.x; e < kUnitM * kUnitN; e += kThreads) {
        const int i = e >> 7, j = e & 127;
        if (i0 + i >= t.mp || j0 + j >= t.np) continue;
        float v = 0.0f;
        if (t.tall) v = turn[j * (kUnitM + 1) + i];
        else if (i0 + i < t.m && j0 + j < t.n) v = src.template get<false>(t, i0 + i, j0 + j);
        f16 hi, lo;
        split(v * inv, hi, lo);
        const int64_t at = (int64_t)(i0 + i) * t.np + j0 + j;
        x[at] = hi;
        y[at] = lo;
    }
}

// ------------------------------------------------------------ products -----
enum Product { kGram, kSquare, kApply, kLastOrth, kLastMuon };

// 16 bytes per lane from `base` + lane_off + off straight into LDS at lds + 16 lane.  A
// buffer access: the tile's address and the row's offset stay in scalar registers and
// all accesses of a side share one vector register (as global accesses they took over
// 100 registers more, and the 256-wide tiles spilled).
__device__ __forceinline__ void copy_to_lds(const f16* base, uint32_t lane_off, uint32_t off, char* lds) {
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, (int)0xFFFFFFFF, 0x00027000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, (int)lane_off, (int)off, 0, 0);
}
// ROWS rows of 64 fp16 (128 bytes) from global memory into LDS, the NW waves'
// share by wave w.  The 16-byte chunk c of row r lies at place c ^ (r & 7) of the
// row, so that 8 lanes that read the same chunk of 8 rows hit 8 different places.
// A tile's rows span at most 256 * 2 * kMostLong bytes, 2.1e9.
__device__ __forceinline__ uint32_t rows_lane_off(uint32_t ld, int lane) {
    return (uint32_t)(lane >> 3) * ld * 2 + (uint32_t)(((lane & 7) ^ (lane >> 3)) * 16);
}
template <int ROWS, int NW>
__device__ __forceinline__ void stage_rows(const f16* base, uint32_t ld, uint32_t lane_off, char* lds, int w) {
#pragma unroll
    for (int q = 0; q < ROWS / 8 / NW; ++q) {
        const uint32_t u = (uint32_t)(q * NW + w);
        copy_to_lds(base, lane_off, u * 16 * ld, lds + u * 1024);
    }
}
// 64 rows (depth) of COLS fp16, for reads that transpose: the 16-byte chunk c of row r
// lies at place c ^ ((r & 3) << 1), so that the 4 rows x 32 bytes that 16 lanes read
// together hit different banks.
template <int COLS, int NW>
__device__ __forceinline__ uint32_t cols_lane_off(uint32_t ld, int lane, int w) {
    constexpr int kPer = COLS / 8, kRows = 64 / kPer;   // chunks of a row; rows of an access
    const int r = lane / kPer, slot = lane % kPer;
    const int key = ((w * kRows + r) & 3) << 1;         // the same in all accesses of the wave
    static_assert(NW * kRows % 4 == 0, "whole turns of the key");
    return (uint32_t)r * ld * 2 + (uint32_t)((slot ^ key) * 16);
}
template <int COLS, int NW>
__device__ __forceinline__ void stage_cols(const f16* base, uint32_t ld, uint32_t lane_off, char* lds, int w) {
    constexpr int kRows = 64 / (COLS / 8);
#pragma unroll
    for (int q = 0; q < kBK / kRows / NW; ++q) {
        const uint32_t u = (uint32_t)(q * NW + w);
        copy_to_lds(base, lane_off, u * kRows * ld * 2, lds + u * 1024);
    }
}
__device__ __forceinline__ f16x8 read_row_frag(const char* lds, int row, int chunk) {
    return *(const f16x8*)(lds + row * 128 + ((chunk ^ (row & 7)) << 4));
}
// Fragment of 16 columns from `col`, lane l's column l % 16, depths k0 + (l / 16) * 8
// + (0..7): two transposing reads, in each of which lane t of 16 brings 4 columns of
// row t / 4 and gets column t of the 4 rows.
template <int COLS>
__device__ __forceinline__ f16x8 read_col_frag(const char* lds, int col, int k0, int lane) {
    const int t = lane & 15, row = k0 + ((lane >> 4) << 3) + (t >> 2);
    const int byte = (col + ((t & 3) << 2)) * 2;
    const char* p = lds + row * (COLS * 2) + (byte ^ ((row & 3) << 5));
    const f16x4 lo = __builtin_bit_cast(f16x4, __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_fp16x4*)p));
    const f16x4 hi = __builtin_bit_cast(f16x4, __builtin_amdgcn_ds_read_tr16_b64_v4f16(
        (lds_fp16x4*)(p + 4 * COLS * 2)));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

constexpr int kTurn = 68;      // floats from row to row of the 16 x 64 block in LDS

// What the wave's lanes wrote to LDS is there for its other lanes.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}
// The block's values by column: lane l gets the 16 rows of column l.
__device__ __forceinline__ void turn_over(char* block, float* at, float* v, int lane) {
#pragma unroll
    for (int e = 0; e < 16; ++e) at[e] = v[e];
    wave_sync();
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = ((const float*)block)[e * kTurn + lane];
}
// 16 elements in one plane, or (plane != 0) in two that lie so far apart.
__device__ __forceinline__ void load_plane(const f16* p, int64_t plane, float* v) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const f16x8 h = *(const f16x8*)(p + 8 * k);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[8 * k + e] = (float)h[e];
    }
    if (plane == 0) return;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const f16x8 l = *(const f16x8*)(p + plane + 8 * k);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[8 * k + e] += (float)l[e];
    }
}
__device__ __forceinline__ void store_plane(f16* p, int64_t plane, const float* v) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        f16x8 h, l;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            f16 hi, lo;
            split(v[8 * k + e], hi, lo);
            h[e] = hi;
            l[e] = lo;
        }
        *(f16x8*)(p + 8 * k) = h;
        if (plane != 0) *(f16x8*)(p + plane + 8 * k) = l;
    }
}
// n <= 16 consecutive elements of a caller's buffer, which may begin at any element.
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
__device__ __forceinline__ void load_f32(const float* p, int n, float* v) {
    if (n == 16) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const f32x4 q = *(const f32x4_a4*)(p + 4 * k);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * k + e] = q[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = e < n ? p[e] : 0.0f;
    }
}
__device__ __forceinline__ void store_f32(void* to, int n, const float* v) {
    float* p = (float*)to;
    if (n == 16) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const f32x4 q = {v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]};
            *(f32x4_a4*)(p + 4 * k) = q;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (e < n) p[e] = v[e];
    }
}
template <int DT>
__device__ __forceinline__ void store_16(void* to, int n, const float* v) {
    uint16_t* p = (uint16_t*)to;
    if (n == 16) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint16_t h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = narrow16(DT, v[8 * k + e]);
            *(u32x4_a2*)(p + 8 * k) = pack8(h);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (e < n) p[e] = narrow16(DT, v[e]);
    }
}

// A tile of one product: T x T, by NW = WM x WN waves.
//   kGram    A = X X^T          rows of X by rows of X
//   kSquare  B = b A + c A A    rows of A by rows of A
//   kApply   X' = a X + B X     rows of B by columns of X; kLast*: into the result
template <int T, int WM, int WN, int OP, int DT>
__global__ void __launch_bounds__(WM * WN * 64, 2)
matrix_product_kernel(Step s, NsConsts ns, int from, int precise, MuonBufs mb, MuonConsts mc) {
    constexpr int NW = WM * WN, FI = T / WM / 16, FJ = T / WN / 16;
    static_assert(FJ == 4, "64 columns to a wave");
    constexpr bool kTri = OP == kGram || OP == kSquare;
    constexpr int kSide = T * kBK * 2;      // bytes of a side's stage
    if (skipped(s.res)) return;
    __shared__ __attribute__((aligned(1024))) char lds0[2 * kSide];
    __shared__ __attribute__((aligned(1024))) char lds1[2 * kSide];
    const Item it = s.items[item_of<32>(blockIdx.x, s.n_items)];
    const Mat& t = s.mats[it.mat];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wi = (w / WN) * (T / WM), wj = (w % WN) * (T / WN);
    const int64_t i0 = (int64_t)it.i * T, j0 = (int64_t)it.j * T;
    const int64_t np = t.np, mp = t.mp;
    const int64_t px = t.plane_x / 2, pa = t.plane_a / 2;
    const f16* x = (const f16*)(s.ws + t.x[from]);
    const f16* a = (const f16*)(s.ws + t.a);
    const f16* b = (const f16*)(s.ws + t.b);
    const f16 *left, *right;
    int64_t left_plane, right_plane, left_ld, right_ld;
    int depth;
    if constexpr (OP == kGram) {
        left = x + i0 * np, right = x + j0 * np;
        left_plane = right_plane = px, left_ld = right_ld = np, depth = (int)np;
    } else if constexpr (OP == kSquare) {
        left = a + i0 * mp, right = a + j0 * mp;
        left_plane = right_plane = pa, left_ld = right_ld = mp, depth = (int)mp;
    } else {
        left = b + i0 * mp, right = x + j0;
        left_plane = pa, right_plane = px, left_ld = mp, right_ld = np, depth = (int)mp;
    }
    f32x4 acc[FI][FJ];
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int j = 0; j < FJ; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const uint32_t left_off = rows_lane_off((uint32_t)left_ld, lane);
    const uint32_t right_off = kTri ? rows_lane_off((uint32_t)right_ld, lane)
                                    : cols_lane_off<T, NW>((uint32_t)right_ld, lane, w);
    const int per = depth / kBK, total = precise ? 3 * per : per;
    auto stage = [&](int k, char* lds) {
        const int seg = k / per, kk = (k - seg * per) * kBK;   // hi hi, hi lo, lo hi
        const f16* l = left + (seg == 2 ? left_plane : 0);
        const f16* r = right + (seg == 1 ? right_plane : 0);
        stage_rows<T, NW>(l + kk, (uint32_t)left_ld, left_off, lds, w);
        if constexpr (kTri) stage_rows<T, NW>(r + kk, (uint32_t)right_ld, right_off, lds + kSide, w);
        else stage_cols<T, NW>(r + kk * right_ld, (uint32_t)right_ld, right_off, lds + kSide, w);
    };
    auto compute = [&](const char* lds) {
#pragma unroll
        for (int ks = 0; ks < kBK / 32; ++ks) {
            f16x8 l[FI], r[FJ];
#pragma unroll
            for (int i = 0; i < FI; ++i)
                l[i] = read_row_frag(lds, wi + i * 16 + (lane & 15), ks * 4 + (lane >> 4));
#pragma unroll
            for (int j = 0; j < FJ; ++j) {
                if constexpr (kTri)
                    r[j] = read_row_frag(lds + kSide, wj + j * 16 + (lane & 15), ks * 4 + (lane >> 4));
                else r[j] = read_col_frag<T>(lds + kSide, wj + j * 16, ks * 32, lane);
            }
#pragma unroll
            for (int i = 0; i < FI; ++i)
#pragma unroll
                for (int j = 0; j < FJ; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(r[j], l[i], acc[i][j], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    float step = 0.0f;                      // lr * alpha
    if constexpr (OP == kLastMuon) {
        double alpha = 1.0;
        if (mc.scaling == ZERO_MUON_ASPECT && t.rows > t.cols)
            alpha = sqrt((double)t.rows / (double)t.cols);
        if (mc.scaling == ZERO_MUON_RMS) alpha = 0.2 * sqrt((double)(t.rows > t.cols ? t.rows : t.cols));
        step = (float)((double)mc.lr * alpha);
    }
    stage(0, lds0);
    __syncthreads();
    for (int k = 0; k + 2 <= total; k += 2) {
        stage(k + 1, lds1);
        compute(lds0);
        __syncthreads();
        if (k + 2 < total) stage(k + 2, lds0);
        compute(lds1);
        __syncthreads();
    }
    if constexpr (T == kBK) {   // larger tiles have an even number of steps
        if (total & 1) {
            compute(lds0);
            __syncthreads();
        }
    }

    // 16 rows of the wave's 64 columns at a time go through LDS, so that what is read
    // and written beside them is 16 consecutive elements per lane
    char* mine = ((w & 1) ? lds1 : lds0) + (w >> 1) * (16 * kTurn * 4);
    const int64_t first = j0 + wj;
#pragma unroll
    for (int i = 0; i < FI; ++i) {
        const int64_t top = i0 + wi + i * 16;
        // lane l holds row l % 16 and 4 columns from (l / 16) * 4 of every fragment
#pragma unroll
        for (int j = 0; j < FJ; ++j)
            *(f32x4*)(mine + ((lane & 15) * kTurn + j * 16 + ((lane >> 4) << 2)) * 4) = acc[i][j];
        wave_sync();
        const int64_t row = top + (lane >> 2), col = first + ((lane & 3) << 4);
        float* at = (float*)mine + (lane >> 2) * kTurn + ((lane & 3) << 4);
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = at[e];
        if constexpr (kTri) {
            f16* out = (f16*)(s.ws + (OP == kGram ? t.a : t.b));
            if constexpr (OP == kGram) {
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] *= kScaleA / (kScaleX * kScaleX);
            } else {
                float h[16];
                load_plane(a + row * mp + col, precise ? pa : 0, h);
                const float p = ns.b * (ns.scale_b / kScaleA);
                const float q = ns.c * (ns.scale_b / (kScaleA * kScaleA));
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = p * h[e] + q * v[e];
            }
            store_plane(out + row * mp + col, precise ? pa : 0, v);
            if (it.i != it.j) {
                turn_over(mine, at, v, lane);
                store_plane(out + (first + lane) * mp + top, precise ? pa : 0, v);
            }
        } else {
            float h[16];
            load_plane(x + row * np + col, px, h);
            const float q = 1.0f / ns.scale_b;
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = ns.a * h[e] + q * v[e];
            if constexpr (OP == kApply) {
                store_plane((f16*)(s.ws + t.x[from ^ 1]) + row * np + col, px, v);
            } else {
                // in memory: row r, 16 consecutive columns from c, or what of them exists
                int64_t r = row, c = col;
                if (t.tall) {
                    turn_over(mine, at, v, lane);
                    r = first + lane, c = top;
                }
                if (r < t.rows && c < t.cols) {
                    const int n = (int)(t.cols - c < 16 ? t.cols - c : 16);
                    if constexpr (OP == kLastOrth) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] *= 1.0f / kScaleX;
                        char* out = (char*)t.dst + (r * t.dst_ld + c) * (t.dst_dtype == ZERO_FP32 ? 4 : 2);
                        if (t.dst_dtype == ZERO_FP32) store_f32(out, n, v);
                        else if (t.dst_dtype == ZERO_FP16) store_16<ZERO_FP16>(out, n, v);
                        else store_16<ZERO_BF16>(out, n, v);
                    } else {
                        const int64_t e0 = t.offset + r * t.cols + c;
                        float p[16];
                        load_f32(mb.master + e0, n, p);
                        const float f = step * (1.0f / kScaleX);
#pragma unroll
                        for (int e = 0; e < 16; ++e) p[e] = p[e] * mc.decay - f * v[e];
                        store_f32(mb.master + e0, n, p);
                        store_16<DT>(mb.p16 + e0, n, p);
                    }
                }
            }
        }
        wave_sync();
        __builtin_amdgcn_sched_barrier(0);
    }
}

// ------------------------------------------------------------ host ---------
int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// The tile of a matrix's products by its shorter side.
int tile_for(int64_t m, int64_t n) {
    (void)n;
    return m <= 64 ? 64 : m <= 1024 ? 128 : 256;
}
// Tiles below the diagonal of a group of matrices, and bytes of its planes, after
// which the next matrix begins another group.
constexpr int64_t kGroupTiles = 1024, kGroupBytes = int64_t(4) << 30;

struct Build {
    std::vector<Group> groups;
    std::vector<Mat> mats;
    std::vector<Item> items;
    int64_t ws = 0;

    bool add(const Mat* in, int64_t count, int tile, bool precise) {
        // longest products first: the last round of blocks is then a short one
        std::vector<Mat> v(in, in + count);
        std::stable_sort(v.begin(), v.end(), [](const Mat& x, const Mat& y) { return x.np > y.np; });
        Group g;
        memset(&g, 0, sizeof g);
        g.tile = tile;
        g.mat0 = (int64_t)mats.size(), g.n_mats = count;
        int64_t at = 0, parts = 0;
        const int planes = precise ? 2 : 1;
        for (Mat& t : v) {
            t.plane_x = (int64_t)t.mp * t.np * 2, t.plane_a = (int64_t)t.mp * t.mp * 2;
            t.x[0] = at, at = up(at + 2 * t.plane_x, 256);
            t.x[1] = at, at = up(at + 2 * t.plane_x, 256);
            t.a = at, at = up(at + planes * t.plane_a, 256);
            t.b = at, at = up(at + planes * t.plane_a, 256);
            const int64_t u = up(t.mp, kUnitM) / kUnitM * (up(t.np, kUnitN) / kUnitN);
            if (u > INT32_MAX) return false;
            t.part0 = parts, t.n_parts = (int32_t)u;
            parts += u;
        }
        g.inv_off = at, at = up(at + 4 * count, 256);
        g.part_off = at, at = up(at + 8 * parts, 256);
        ws = std::max(ws, at);
        g.unit0 = (int64_t)items.size();
        for (int64_t k = 0; k < count; ++k)
            for (int64_t i = 0; i * kUnitM < v[k].mp; ++i)
                for (int64_t j = 0; j * kUnitN < v[k].np; ++j) item(g.mat0 + k, i, j);
        g.n_units = (int64_t)items.size() - g.unit0;
        g.tri0 = (int64_t)items.size();
        for (int64_t k = 0; k < count; ++k)
            for (int64_t i = 0; i * tile < v[k].mp; ++i)
                for (int64_t j = 0; j <= i; ++j) item(g.mat0 + k, i, j);
        g.n_tri = (int64_t)items.size() - g.tri0;
        g.full0 = (int64_t)items.size();
        // bands of 4 rows of tiles, column by column: the blocks that run together
        // share rows of B and columns of X
        for (int64_t k = 0; k < count; ++k)
            for (int64_t i = 0; i * tile < v[k].mp; i += 4)
                for (int64_t j = 0; j * tile < v[k].np; ++j)
                    for (int64_t q = i; q < i + 4 && q * tile < v[k].mp; ++q) item(g.mat0 + k, q, j);
        g.n_full = (int64_t)items.size() - g.full0;
        if (g.n_units > kMaxLaunchBlocks || g.n_full > kMaxLaunchBlocks) return false;
        mats.insert(mats.end(), v.begin(), v.end());
        groups.push_back(g);
        return true;
    }
    void item(int64_t mat, int64_t i, int64_t j) {
        items.push_back(Item{(uint32_t)mat, (uint16_t)i, (uint16_t)j});
    }
    int make(std::vector<Mat>& in, bool precise) {
        for (Mat& t : in) {
            t.tall = t.rows > t.cols;
            t.m = std::min(t.rows, t.cols), t.n = std::max(t.rows, t.cols);
        }
        for (const int tile : {64, 128, 256}) {
            std::vector<Mat> v;
            int64_t tiles = 0, bytes = 0;
            for (Mat& t : in) {
                if (t.m == 0 || tile_for(t.m, t.n) != tile) continue;
                t.mp = (int32_t)up(t.m, tile), t.np = (int32_t)up(t.n, tile);
                const int64_t q = t.mp / tile;
                v.push_back(t);
                tiles += q * (q + 1) / 2;
                bytes += 8 * (int64_t)t.mp * t.np + 8 * (int64_t)t.mp * t.mp;
                if (tiles >= kGroupTiles || bytes >= kGroupBytes) {
                    if (!add(v.data(), (int64_t)v.size(), tile, precise)) return ZERO_ERANGE;
                    v.clear();
                    tiles = bytes = 0;
                }
            }
            if (!v.empty() && !add(v.data(), (int64_t)v.size(), tile, precise)) return ZERO_ERANGE;
        }
        return ZERO_OK;
    }
    Head head() const {
        Head h;
        h.magic = kMagic;
        h.n_groups = (int64_t)groups.size();
        h.groups_off = sizeof(Head);
        h.mats_off = up(h.groups_off + (int64_t)(groups.size() * sizeof(Group)), 256);
        h.items_off = up(h.mats_off + (int64_t)(mats.size() * sizeof(Mat)), 256);
        h.bytes = up(h.items_off + (int64_t)(items.size() * sizeof(Item)), 256);
        return h;
    }
    void write(char* to) const {
        const Head h = head();
        memset(to, 0, (size_t)h.bytes);
        memcpy(to, &h, sizeof h);
        if (!groups.empty()) memcpy(to + h.groups_off, groups.data(), groups.size() * sizeof(Group));
        if (!mats.empty()) memcpy(to + h.mats_off, mats.data(), mats.size() * sizeof(Mat));
        if (!items.empty()) memcpy(to + h.items_off, items.data(), items.size() * sizeof(Item));
    }
};

int check_sides(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0) return ZERO_EINVAL;
    if (std::max(rows, cols) > kMostLong || std::min(rows, cols) > kMostShort) return ZERO_ERANGE;
    return ZERO_OK;
}
bool valid_type(int32_t dt) { return dt == ZERO_FP32 || dt == ZERO_FP16 || dt == ZERO_BF16; }

// The bytes that a matrix's rows lie in, as rows of `row` bytes every `pitch`.
struct Span {
    uintptr_t at, end, row, pitch;
    bool write;
    int64_t owner;
};
// Whether two spans share a byte.  Column blocks of one buffer (the same pitch)
// interleave without sharing any.
bool share(const Span& x, const Span& y) {
    if (x.end <= y.at || y.end <= x.at) return false;
    if (x.pitch != y.pitch) return true;
    const Span &lo = x.at <= y.at ? x : y, &hi = x.at <= y.at ? y : x;
    const uintptr_t d = (hi.at - lo.at) % lo.pitch;
    return d < lo.row || d + hi.row > lo.pitch;
}

int build_entries(const zero_matrix_entry* e, int64_t n, Build& b, bool precise, int64_t* numel) {
    std::vector<Mat> v;
    std::vector<Span> spans;
    *numel = 0;
    for (int64_t k = 0; k < n; ++k) {
        const zero_matrix_entry& x = e[k];
        if (const int rc = check_sides(x.rows, x.cols)) return rc;
        if (!valid_type(x.src_dtype) || !valid_type(x.dst_dtype)) return ZERO_EINVAL;
        if (x.rows == 0 || x.cols == 0) continue;
        const uintptr_t sb = x.src_dtype == ZERO_FP32 ? 4 : 2, db = x.dst_dtype == ZERO_FP32 ? 4 : 2;
        const uintptr_t sp = (uintptr_t)x.src, dp = (uintptr_t)x.dst;
        if (!sp || !dp || sp % sb || dp % db) return ZERO_EINVAL;
        if (x.src_ld < x.cols || x.dst_ld < x.cols) return ZERO_EINVAL;
        Span s[2] = {{sp, 0, (uintptr_t)x.cols * sb, 0, false, k}, {dp, 0, (uintptr_t)x.cols * db, 0, true, k}};
        const int64_t lds[2] = {x.src_ld, x.dst_ld};
        const uintptr_t size[2] = {sb, db};
        for (int q = 0; q < 2; ++q) {
            uintptr_t extent;
            if (__builtin_mul_overflow((uintptr_t)lds[q], size[q], &s[q].pitch) ||
                __builtin_mul_overflow(s[q].pitch, (uintptr_t)(x.rows - 1), &extent) ||
                __builtin_add_overflow(extent, s[q].row, &extent) ||
                __builtin_add_overflow(s[q].at, extent, &s[q].end) || s[q].end > (uintptr_t)INT64_MAX)
                return ZERO_ERANGE;
            spans.push_back(s[q]);
        }
        Mat t;
        memset(&t, 0, sizeof t);
        t.src = x.src, t.dst = x.dst;
        t.src_ld = x.src_ld, t.dst_ld = x.dst_ld;
        t.rows = (int32_t)x.rows, t.cols = (int32_t)x.cols;
        t.src_dtype = x.src_dtype, t.dst_dtype = x.dst_dtype;
        v.push_back(t);
        *numel += x.rows * x.cols;
    }
    // No result overlaps another result, nor a matrix other than its own in the same
    // place.  Spans sorted by their beginning; those still open are looked at.
    std::sort(spans.begin(), spans.end(), [](const Span& x, const Span& y) { return x.at < y.at; });
    std::vector<Span> open;
    for (const Span& s : spans) {
        size_t kept = 0;
        for (const Span& o : open) {
            if (o.end <= s.at) continue;
            open[kept++] = o;
        }
        open.resize(kept);
        for (const Span& o : open) {
            if (!s.write && !o.write) continue;
            if (s.owner == o.owner && s.at == o.at && s.pitch == o.pitch && s.row == o.row) continue;
            if (share(s, o)) return ZERO_EINVAL;
        }
        open.push_back(s);
    }
    return b.make(v, precise);
}

int build_ranges(const zero_matrix_range* r, int64_t n, Build& b, bool precise, int64_t* numel,
                 int64_t* extent) {
    std::vector<Mat> v;
    std::vector<std::pair<int64_t, int64_t>> spans;
    *numel = *extent = 0;
    for (int64_t k = 0; k < n; ++k) {
        if (const int rc = check_sides(r[k].rows, r[k].cols)) return rc;
        if (r[k].offset < 0) return ZERO_EINVAL;
        if (r[k].rows == 0 || r[k].cols == 0) continue;
        const int64_t count = r[k].rows * r[k].cols;   // at most 2^38
        int64_t end;
        if (__builtin_add_overflow(r[k].offset, count, &end) || end > INT64_MAX / 4) return ZERO_ERANGE;
        spans.emplace_back(r[k].offset, end);
        Mat t;
        memset(&t, 0, sizeof t);
        t.offset = r[k].offset;
        t.rows = (int32_t)r[k].rows, t.cols = (int32_t)r[k].cols;
        t.src_ld = t.dst_ld = t.cols;
        v.push_back(t);
        *numel += count;
        *extent = std::max(*extent, end);
    }
    std::sort(spans.begin(), spans.end());
    for (size_t k = 1; k < spans.size(); ++k)
        if (spans[k].first < spans[k - 1].second) return ZERO_EINVAL;
    return b.make(v, precise);
}

enum { kKindEntries = 1, kKindRanges = 2 };

int fill_plan(const Build& b, int32_t kind, int64_t n, int64_t numel, int64_t extent, bool precise,
              zero_matrix_plan* plan) {
    memset(plan, 0, sizeof *plan);
    plan->n_matrices = n, plan->numel = numel, plan->extent = extent;
    plan->table_bytes = b.head().bytes;
    plan->workspace_bytes = b.ws;
    plan->kind = kind, plan->precise = precise ? 1 : 0;
    return ZERO_OK;
}
bool same_plan(const zero_matrix_plan& x, const zero_matrix_plan& y) {
    return x.n_matrices == y.n_matrices && x.numel == y.numel && x.extent == y.extent &&
           x.table_bytes == y.table_bytes && x.workspace_bytes == y.workspace_bytes &&
           x.kind == y.kind && x.precise == y.precise;
}

template <typename F>
int guarded(F&& f) {
    try {
        return f();
    } catch (const std::bad_alloc&) {
        return ZERO_ERANGE;
    } catch (const std::length_error&) {
        return ZERO_ERANGE;
    }
}

// Bounds of the singular values through the steps, from 1: the largest value that the
// polynomial takes between 0 and the last bound.  Also a bound of B's eigenvalues.
// Sampled at 4096 points with the second-order error added.
bool ns_bounds(const zero_newton_schulz& ns, double* most_b) {
    const double a = ns.a, b = ns.b, c = ns.c;
    double r = 1.0, top_b = 0.0;
    for (int k = 0; k < ns.steps; ++k) {
        const int n = 4096;
        double top = 0.0;
        for (int q = 0; q <= n; ++q) {
            const double x = r * q / n, l = x * x;
            const double e = b * l + c * l * l;
            top_b = std::max(top_b, fabs(e));
            top = std::max(top, fabs((a + e) * x));
        }
        const double h = r / n;
        top += h * h / 8 * (6 * fabs(b) * r + 20 * fabs(c) * r * r * r);
        if (!(top <= kMostSigma)) return false;
        r = std::max(top, 1e-3);
    }
    *most_b = top_b * 1.1 + 1e-3;
    return true;
}

int ns_consts(const zero_newton_schulz* ns, NsConsts* out) {
    if (!ns || ns->steps < 1 || ns->steps > 64) return ZERO_EINVAL;
    if (!isfinite(ns->a) || !isfinite(ns->b) || !isfinite(ns->c) || !isfinite(ns->eps) ||
        !(ns->eps >= 1e-30f))
        return ZERO_EINVAL;
    double most = 0.0;
    if (!ns_bounds(*ns, &most)) return ZERO_EINVAL;
    out->a = ns->a, out->b = ns->b, out->c = ns->c, out->eps = ns->eps;
    // the power of two that takes the bound to at most 2^15, and B to at least A's scale / 2^14
    int e = 0;
    frexp(most, &e);
    e = 15 - e;
    if (e < 0) return ZERO_EINVAL;
    if (e > 14) e = 14;
    out->scale_b = ldexpf(1.0f, e);
    return ZERO_OK;
}

template <int T, int WM, int WN, int DT>
int run_steps(const Step& base, const Group& g, const Item* items, const NsConsts& ns, int steps,
              int precise, bool muon, const MuonBufs& mb, const MuonConsts& mc, hipStream_t stream) {
    Step tri = base, full = base;
    tri.items = items + g.tri0, tri.n_items = g.n_tri;
    full.items = items + g.full0, full.n_items = g.n_full;
    constexpr int kLanes = WM * WN * 64;
    for (int k = 0; k < steps; ++k) {
        const int from = k & 1;
        int rc = launch_shape(matrix_product_kernel<T, WM, WN, kGram, 0>, g.n_tri, kLanes, 0, stream, tri,
                              ns, from, precise, mb, mc);
        if (rc == ZERO_OK)
            rc = launch_shape(matrix_product_kernel<T, WM, WN, kSquare, 0>, g.n_tri, kLanes, 0, stream, tri,
                              ns, from, precise, mb, mc);
        if (rc == ZERO_OK)
            rc = k + 1 < steps
                ? launch_shape(matrix_product_kernel<T, WM, WN, kApply, 0>, g.n_full, kLanes, 0, stream,
                               full, ns, from, precise, mb, mc)
                : muon ? launch_shape(matrix_product_kernel<T, WM, WN, kLastMuon, DT>, g.n_full, kLanes, 0,
                                      stream, full, ns, from, precise, mb, mc)
                       : launch_shape(matrix_product_kernel<T, WM, WN, kLastOrth, 0>, g.n_full, kLanes, 0,
                                      stream, full, ns, from, precise, mb, mc);
        if (rc != ZERO_OK) return rc;
    }
    return ZERO_OK;
}

// Every group in turn, on one stream: they share the workspace.
template <int DT, typename Source>
int run_groups(const char* host, const char* table, const NsConsts& ns, int steps, int precise, bool muon,
               Source src, const MuonBufs& mb, const MuonConsts& mc, const zero_step_result* res, char* ws,
               hipStream_t stream) {
    Head h;
    memcpy(&h, host, sizeof h);
    const Item* items = (const Item*)(table + h.items_off);
    for (int64_t k = 0; k < h.n_groups; ++k) {
        Group g;
        memcpy(&g, host + h.groups_off + k * (int64_t)sizeof(Group), sizeof g);
        Step s;
        s.mats = (const Mat*)(table + h.mats_off);
        s.items = items + g.unit0, s.n_items = g.n_units;
        s.ws = ws, s.res = res;
        s.inv_off = g.inv_off, s.part_off = g.part_off;
        int rc = launch(matrix_norm_kernel<Source>, g.n_units, 0, stream, s, src);
        if (rc != ZERO_OK) return rc;
        Step f = s;
        f.mats = s.mats + g.mat0;
        rc = launch(matrix_factor_kernel, g.n_mats, 0, stream, f, ns.eps);
        if (rc != ZERO_OK) return rc;
        rc = launch(matrix_init_kernel<Source>, g.n_units, 0, stream, s, g.mat0, src);
        if (rc != ZERO_OK) return rc;
        rc = g.tile == 64 ? run_steps<64, 4, 1, DT>(s, g, items, ns, steps, precise, muon, mb, mc, stream)
           : g.tile == 128 ? run_steps<128, 2, 2, DT>(s, g, items, ns, steps, precise, muon, mb, mc, stream)
                           : run_steps<256, 2, 4, DT>(s, g, items, ns, steps, precise, muon, mb, mc, stream);
        if (rc != ZERO_OK) return rc;
    }
    return ZERO_OK;
}

// A plan with its table, as every call gets them.
int check_call(const zero_matrix_plan* plan, int32_t kind, const void* host, const void* table,
               const void* ws, size_t ws_bytes) {
    if (!plan || plan->kind != kind || !host || !table || (uintptr_t)table % 16) return ZERO_EINVAL;
    Head h;
    memcpy(&h, host, sizeof h);
    if (h.magic != kMagic || h.bytes != plan->table_bytes) return ZERO_EINVAL;
    if (h.n_groups == 0) return ZERO_OK;
    if (!ws || (uintptr_t)ws % 256 || ws_bytes < (size_t)plan->workspace_bytes) return ZERO_EINVAL;
    return ZERO_OK;
}

}  // namespace

extern "C" {

int zero_matrix_plan_init(const zero_matrix_entry* entries, int64_t n_matrices, int32_t precise,
                          zero_matrix_plan* plan) {
    if (!plan || n_matrices < 0 || (n_matrices > 0 && !entries)) return ZERO_EINVAL;
    return guarded([&] {
        Build b;
        int64_t numel;
        const int rc = build_entries(entries, n_matrices, b, precise != 0, &numel);
        return rc != ZERO_OK ? rc : fill_plan(b, kKindEntries, n_matrices, numel, 0, precise != 0, plan);
    });
}

int zero_matrix_plan_table(const zero_matrix_entry* entries, const zero_matrix_plan* plan, void* table) {
    if (!plan || !table || plan->kind != kKindEntries || plan->n_matrices < 0 ||
        (plan->n_matrices > 0 && !entries))
        return ZERO_EINVAL;
    return guarded([&] {
        Build b;
        int64_t numel;
        const int rc = build_entries(entries, plan->n_matrices, b, plan->precise != 0, &numel);
        if (rc != ZERO_OK) return rc;
        zero_matrix_plan again;
        fill_plan(b, kKindEntries, plan->n_matrices, numel, 0, plan->precise != 0, &again);
        if (!same_plan(again, *plan)) return (int)ZERO_EINVAL;
        b.write((char*)table);
        return (int)ZERO_OK;
    });
}

int zero_muon_plan_init(const zero_matrix_range* ranges, int64_t n_matrices, int32_t precise,
                        zero_matrix_plan* plan) {
    if (!plan || n_matrices < 0 || (n_matrices > 0 && !ranges)) return ZERO_EINVAL;
    return guarded([&] {
        Build b;
        int64_t numel, extent;
        const int rc = build_ranges(ranges, n_matrices, b, precise != 0, &numel, &extent);
        return rc != ZERO_OK ? rc
                             : fill_plan(b, kKindRanges, n_matrices, numel, extent, precise != 0, plan);
    });
}

int zero_muon_plan_table(const zero_matrix_range* ranges, const zero_matrix_plan* plan, void* table) {
    if (!plan || !table || plan->kind != kKindRanges || plan->n_matrices < 0 ||
        (plan->n_matrices > 0 && !ranges))
        return ZERO_EINVAL;
    return guarded([&] {
        Build b;
        int64_t numel, extent;
        const int rc = build_ranges(ranges, plan->n_matrices, b, plan->precise != 0, &numel, &extent);
        if (rc != ZERO_OK) return rc;
        zero_matrix_plan again;
        fill_plan(b, kKindRanges, plan->n_matrices, numel, extent, plan->precise != 0, &again);
        if (!same_plan(again, *plan)) return (int)ZERO_EINVAL;
        b.write((char*)table);
        return (int)ZERO_OK;
    });
}

int zero_orthogonalize(const zero_matrix_plan* plan, const void* host_table, const void* table,
                       const zero_newton_schulz* ns, void* workspace, size_t workspace_bytes,
                       hipStream_t stream) {
    NsConsts c;
    if (const int rc = ns_consts(ns, &c)) return rc;
    if (const int rc = check_call(plan, kKindEntries, host_table, table, workspace, workspace_bytes)) return rc;
    const MuonBufs mb = {nullptr, nullptr, nullptr, nullptr};
    const MuonConsts mc = {0, 0, 0, 0, 0, 0};
    return run_groups<0>((const char*)host_table, (const char*)table, c, ns->steps, plan->precise, false,
                         OrthSource{}, mb, mc, nullptr, (char*)workspace, stream);
}

int zero_muon_step(float* master, float* momentum, void* param16, const void* grad16, int32_t dtype,
                   const zero_matrix_plan* plan, const void* host_table, const void* table,
                   const zero_muon_hparams* hp, const zero_step_result* res, void* workspace,
                   size_t workspace_bytes, hipStream_t stream) {
    NsConsts c;
    if (!hp || !res || !valid_dtype(dtype)) return ZERO_EINVAL;
    if (!isfinite(hp->lr) || !isfinite(hp->momentum) || !isfinite(hp->weight_decay) ||
        isnan(hp->max_grad_norm) || hp->scaling < ZERO_MUON_NONE || hp->scaling > ZERO_MUON_RMS)
        return ZERO_EINVAL;
    if (const int rc = ns_consts(&hp->ns, &c)) return rc;
    if (const int rc = check_call(plan, kKindRanges, host_table, table, workspace, workspace_bytes)) return rc;
    if (plan->numel == 0) return ZERO_OK;
    if (!master || !momentum || !param16 || !grad16) return ZERO_EINVAL;
    if ((uintptr_t)master % 4 || (uintptr_t)momentum % 4 || (uintptr_t)param16 % 2 ||
        (uintptr_t)grad16 % 2 || (uintptr_t)res % 8)
        return ZERO_EINVAL;
    const MuonBufs mb = {master, momentum, (uint16_t*)param16, (const uint16_t*)grad16};
    MuonConsts mc;
    mc.momentum = hp->momentum;
    mc.decay = (float)(1.0 - (double)hp->lr * (double)hp->weight_decay);
    mc.lr = hp->lr, mc.max_norm = hp->max_grad_norm;
    mc.nesterov = hp->nesterov != 0, mc.scaling = hp->scaling;
    const char *host = (const char*)host_table, *dev = (const char*)table;
    if (dtype == ZERO_FP16)
        return run_groups<ZERO_FP16>(host, dev, c, hp->ns.steps, plan->precise, true,
                                     MuonSource<ZERO_FP16>{mb, mc, 0, 0}, mb, mc, res, (char*)workspace,
                                     stream);
    return run_groups<ZERO_BF16>(host, dev, c, hp->ns.steps, plan->precise, true,
                                 MuonSource<ZERO_BF16>{mb, mc, 0, 0}, mb, mc, res, (char*)workspace, stream);
}

}  // extern "C"
