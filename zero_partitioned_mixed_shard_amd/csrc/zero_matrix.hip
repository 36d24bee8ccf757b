// zero_matrix.hip -- steps of whole matrices: orthogonalisation by Newton-Schulz
// products (zero_orthogonalize) and the Muon step of an owner's matrices
// (zero_muon_step), over a plan of matrices of any sizes.
//
// Mathematics.  X is the matrix in its wide form (m <= n; a tall matrix is
// transposed on the way in and out), divided by its Frobenius norm; then `steps`
// times
//     A = X X^T,   B = b A + c A A,   X <- a X + B X,
// which applies the polynomial a x + b x^3 + c x^5 to the singular values and
// leaves the singular vectors.  A and what is made of it are polynomials of one symmetric
// matrix, so they commute and are symmetric: only the tiles on and below the diagonal are
// computed, and written twice.  A step is 3 m^2 n + m^3 operations (4 m^2 n + 2 m^3 without
// the symmetry); two steps to a pass over X (pairs_for) are 3 m^2 n + 5 m^3.
//
// Bounds.  Large matrices are bound by the matrix cores, at the clock that their power
// leaves: a product with X of 8192 x 28672 runs at 1235 TFLOP/s (1324 in its loop), where the
// library's of 8192^3 reaches 1517.  Of matrices of 1024 to 2048 the tiles' ends weigh (a
// quarter of the time at a depth of 2048: X's two parts and the planes through HBM), of
// smaller ones the launches.
//
// Numerics.  The products run on the matrix cores in fp16 with fp32 sums.  fp16 has
// three bits more than bf16 at the same rate, and its range is enough here: a
// matrix's entries are bounded by its largest singular value, which the host bounds
// for the given coefficients (at most 1.75), so X is kept times 2^15 and A times
// 2^14 and nothing overflows, while entries down to 2^-29 stay normal.  X is kept in
// two parts, hi = fp16(x) and lo = fp16(x - hi).  A direction of small singular values is
// multiplied by a in every step (485 times in 5 steps), and so would be the rounding of X:
// the linear term a X takes both parts, the products hi alone, but for what is large on the
// planes' diagonals: what these lose in rounding, and their product with lo, are added in
// the tiles' ends to first order.  Relative error of the result (2-norm) against 64 bits, for
// the usual coefficients: 2e-4 to 1e-3 for matrices of full rank, or of low rank with some
// percent of noise.  Where many directions have no part the planes are not near a multiple of
// the identity, and the roundings off their diagonals count: up to 0.06 / sqrt(m) of exactly
// or almost low rank or of two levels (3.6e-3 at 65 x 200, 1.4e-3 at 1024 x 1024), 0.08 of one
// direction (8.5e-3 at 65 x 20000), 0.1 with two steps to a pass (1.6e-3 at 2048 x 4096).
// Where all entries are alike so are their roundings: 8e-3, in pairs 2.1e-2.  Without lo a
// matrix of almost rank 1 would be off by 0.12, in bf16 by 1.
// With `precise` A, B and X have two parts and every product is lo hi + hi lo + hi hi, three
// times the matrix work: 1e-6 to 5e-6, up to 2e-5 of low rank; of rank 1 to 16, whose result
// is small beside what the other directions make of X's last bits, more (16384 x 16384 of rank
// 1 4e-4, of rank 4 1.4e-4, of rank 16 8e-5), and 4e-4 where all entries are alike (hi hi first
// would be 6.7e-6 of full rank and not 2.7e-6, 9.5e-4 and not 4e-4, 5.8e-3 and not 4e-4).

#include <math.h>
#include <string.h>

#include <algorithm>
#include <new>
#include <stdexcept>
#include <utility>
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
// What the steps may multiply an error of X by: X is rounded to 22 bits.
constexpr double kMostGrowth = 1 << 20;
constexpr int64_t kMostLong = 4194240, kMostShort = 65536;   // sides of a matrix
constexpr int kBK = 32;                    // depth of a stage: 64 bytes of a row
constexpr int kUnitM = 64, kUnitN = 128;   // elements of a unit of the streaming passes

// Square planes of a matrix (A, B and a third) and their vectors.
constexpr int kPlanes = 3;

// A matrix of the plan, as the kernels read it.
struct Mat {
    const void* src;            // orthogonalize: the matrix and its result
    void* dst;
    int64_t offset;             // muon: its first element in the shard
    int64_t src_ld, dst_ld;     // elements between rows
    int64_t x[2], p[kPlanes];   // byte offsets in the workspace: X, two of it; the planes
    int64_t r[kPlanes];         // the planes' diagonals, fp32: what they lost in rounding, and whole
    int64_t plane_x, plane_a;   // bytes of a part of X, and of a plane
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
// Tiles of a product: the last ones, of a round that would leave most of the device
// idle, are each cut along the depth into `parts`.
struct Cut {
    int64_t whole;
    int32_t parts, pad;
};
// Matrices that go through the steps together.
struct Group {
    int64_t mat0, n_mats, unit0, n_units, tri0, n_tri, full0, n_full;
    Cut gram, square, apply;
    int64_t inv_off, part_off;  // the norms' factors and partials in the workspace
    int64_t sums_off;           // partial sums of cut tiles
    int32_t tile, pairs;        // pairs: two steps to a pass over X
};
struct Head {
    uint64_t magic;
    int64_t n_groups, groups_off, mats_off, items_off, bytes;
};
constexpr uint64_t kMagic = 0x7a65726f6d617431ull;

static_assert(kUnitM * kUnitN == 8192, "4 times 8 elements for each of 256 lanes");

// What a call passes to every kernel.
struct Step {
    const Mat* mats;
    const Item* items;      // of the launch
    int64_t n_items;
    char* ws;
    const zero_step_result* res;   // NULL: orthogonalize
    int64_t inv_off, part_off, sums_off;
};
// One product.  Its planes hold values times a power of two; the factors undo that.
//   kGram    out = c X X^T
//   kSquare  out = p P + q Q + c P Q     (P and Q commute: the product is symmetric)
//   kApply   X' = p X + c P X
struct Product {
    int32_t from;           // which X
    int32_t p, q, out;      // planes
    int32_t lower;          // p's lower part counts in its own term (kGram: is written)
    float fp, fq, fc;
    Cut cut;
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

// lr * alpha of a matrix.
__device__ __forceinline__ float muon_step(const Mat& t, const MuonConsts& mc) {
    double alpha = 1.0;
    if (mc.scaling == ZERO_MUON_ASPECT && t.rows > t.cols) alpha = sqrt((double)t.rows / (double)t.cols);
    if (mc.scaling == ZERO_MUON_RMS) alpha = 0.2 * sqrt((double)(t.rows > t.cols ? t.rows : t.cols));
    return (float)((double)mc.lr * alpha);
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
    asm("" : "+v"(f));      // rounded to fp32 before (the compiler would skip that)
    if (dt == ZERO_FP16) return __builtin_bit_cast(uint16_t, (f16)f);
    const uint32_t u = __float_as_uint(f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((u >> 16) | 0x0040u);
    return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}
__device__ __forceinline__ float load_elem(const void* p, int64_t e, int dt) {
    return dt == ZERO_FP32 ? ((const float*)p)[e] : widen16(dt, ((const uint16_t*)p)[e]);
}

__device__ __forceinline__ void store_elem(void* p, int64_t e, int dt, float v) {
    if (dt == ZERO_FP32) ((float*)p)[e] = v;
    else ((uint16_t*)p)[e] = narrow16(dt, v);
}

// 8 consecutive elements of a buffer, which may begin at any element.
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
__device__ __forceinline__ void load8_f32(const float* p, float* v) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const f32x4 q = *(const f32x4_a4*)(p + 4 * k);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * k + e] = q[e];
    }
}
__device__ __forceinline__ void load8_16(int dt, const uint16_t* p, float* v) {
    const u32x4 q = *(const u32x4_a2*)p;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = widen16(dt, half_of(q, e));
}

// ------------------------------------------------------------ norm, init ----
// 8 elements of the update from (row, col) of a matrix, of which n exist (the others are
// 0).  Source of the two streaming passes: orthogonalize reads the matrix, the Muon step
// makes the update of gradient and momentum (and stores the momentum in the first pass;
// the second makes the same value again from what was stored).
struct OrthSource {
    __device__ void begin(const Step&) {}
    template <bool FIRST>
    __device__ __forceinline__ void get(const Mat& t, int64_t row, int64_t col, int n, float* v) const {
        const int64_t at = row * t.src_ld + col;
        if (n == 8) {
            if (t.src_dtype == ZERO_FP32) load8_f32((const float*)t.src + at, v);
            else load8_16(t.src_dtype, (const uint16_t*)t.src + at, v);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = e < n ? load_elem(t.src, at + e, t.src_dtype) : 0.0f;
        }
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
    __device__ __forceinline__ void get(const Mat& t, int64_t row, int64_t col, int n, float* v) const {
        const int64_t at = t.offset + row * t.cols + col;
        float g[8], mo[8];
        if (n == 8) {
            load8_16(DT, p.g16 + at, g);
            load8_f32(p.momentum + at, mo);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                g[e] = e < n ? widen16(DT, p.g16[at + e]) : 0.0f;
                mo[e] = e < n ? p.momentum[at + e] : 0.0f;
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            g[e] = g[e] * inv * coef;
            if (FIRST) mo[e] = c.momentum * mo[e] + g[e];
            v[e] = c.nesterov ? g[e] + c.momentum * mo[e] : mo[e];
            if (e >= n) v[e] = 0.0f;
        }
        if (FIRST) {
            if (n == 8) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const f32x4 q = {mo[4 * k], mo[4 * k + 1], mo[4 * k + 2], mo[4 * k + 3]};
                    *(f32x4_a4*)(p.momentum + at + 4 * k) = q;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < n) p.momentum[at + e] = mo[e];
            }
        }
    }
};

// A unit is 64 x 128 elements of the wide form: 64 rows of 128 columns in memory, or of
// a tall matrix 128 rows of 64.  A lane has 8 columns of a row, 4 times; lane_at gives
// its q-th row and first column in memory, and how many of the 8 exist.
__device__ __forceinline__ int lane_at(const Mat& t, const Item& it, int q, int64_t& row, int64_t& col) {
    const int lanes = t.tall ? kUnitM / 8 : kUnitN / 8;       // to a row
    const int r = (int)threadIdx.x / lanes + q * (kThreads / lanes);
    row = (int64_t)(t.tall ? it.j * kUnitN : it.i * kUnitM) + r;
    col = (int64_t)(t.tall ? it.i * kUnitM : it.j * kUnitN) + (int)threadIdx.x % lanes * 8;
    if (row >= t.rows || col >= t.cols) return 0;
    return t.cols - col < 8 ? (int)(t.cols - col) : 8;
}
constexpr int kQuarters = kUnitM * kUnitN / 8 / kThreads;

// First pass: the sum of squares of every unit's elements, in fp64.
template <typename Source>
__global__ void __launch_bounds__(kThreads)
matrix_norm_kernel(Step s, Source src) {
    if (skipped(s.res)) return;
    src.begin(s);
    const int64_t idx = item_of<8>(blockIdx.x, s.n_items);
    const Item it = s.items[idx];
    const Mat t = s.mats[it.mat];
    double sum = 0.0;
#pragma unroll
    for (int q = 0; q < kQuarters; ++q) {
        int64_t row, col;
        const int n = lane_at(t, it, q, row, col);
        if (n == 0) continue;
        float v[8];
        src.template get<true>(t, row, col, n, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fma((double)v[e], (double)v[e], sum);
    }
    __shared__ double part[kThreads / 64];
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0)
        ((double*)(s.ws + s.part_off))[idx] = (part[0] + part[1]) + (part[2] + part[3]);
}

// A factor of a matrix's elements as two, the first a power of two: of a norm near the end of
// fp32's range or beyond it the factor itself would be subnormal, and lose bits.  (v * 2^-64 is
// exact, or of an element that is 0 beside the norm.)
__device__ __forceinline__ void store_factor(float* to, double by) {
    const bool large = by < 0x1p-64;
    to[0] = large ? 0x1p-64f : 1.0f;
    to[1] = (float)(large ? by * 0x1p64 : by);
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
        store_factor((float*)(s.ws + s.inv_off) + 2 * blockIdx.x, (double)kScaleX / (norm + (double)eps));
    }
}

// v is made a value of its own first: the compiler would otherwise round the product or
// sum that it is once, straight to fp16, in one of hi's uses and by way of fp32 in another.
__device__ __forceinline__ void split(float v, f16& hi, f16& lo) {
    asm("" : "+v"(v));
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
    const float* inv = (const float*)(s.ws + s.inv_off) + 2 * (it.mat - mat0);
    const float inv0 = inv[0], inv1 = inv[1];
    f16* x = (f16*)(s.ws + t.x[0]);
    const int64_t lower = t.plane_x / 2;
    float v[kQuarters][8];
#pragma unroll
    for (int q = 0; q < kQuarters; ++q) {
        int64_t row, col;
        const int n = lane_at(t, it, q, row, col);
        if (n > 0) {
            src.template get<false>(t, row, col, n, v[q]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[q][e] = 0.0f;
        }
    }
    if (t.tall) {
#pragma unroll
        for (int q = 0; q < kQuarters; ++q)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                turn[((int)threadIdx.x / 8 + q * 32) * (kUnitM + 1) + (int)threadIdx.x % 8 * 8 + e] = v[q][e];
        __syncthreads();
    }
    // lane: 8 columns of a row of the wide form
#pragma unroll
    for (int q = 0; q < kQuarters; ++q) {
        const int i = (int)threadIdx.x / 16 + q * 16, j = (int)threadIdx.x % 16 * 8;
        if (t.tall) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[q][e] = turn[(j + e) * (kUnitM + 1) + i];
        }
        f16x8 hi, lo;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            f16 h, l;
            split(v[q][e] * inv0 * inv1, h, l);
            hi[e] = h;
            lo[e] = l;
        }
        const int64_t at = ((int64_t)it.i * kUnitM + i) * t.np + (int64_t)it.j * kUnitN + j;
        *(f16x8*)(x + at) = hi;
        *(f16x8*)(x + lower + at) = lo;
    }
}

// ------------------------------------------------------------ products -----
// 16 bytes per lane from `base` + lane_off + off straight into LDS at lds + 16 lane.  A
// buffer access: the tile's address and the row's offset stay in scalar registers and
// all accesses of a side share one vector register (as global accesses they took over
// 100 registers more, and the 256-wide tiles spilled).
__device__ __forceinline__ void copy_to_lds(const f16* base, uint32_t lane_off, uint32_t off, char* lds) {
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, (int)0xFFFFFFFF, 0x00027000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, (int)lane_off, (int)off, 0, 0);
}
// ROWS rows of 32 fp16 (64 bytes) from global memory into LDS, the NW waves' share by
// wave w.  The 16-byte chunk c of row r lies at place c ^ ((r >> 1) & 3) of the row, so
// that 8 lanes that read the same chunk of 8 rows hit 8 different places of 128 bytes.
// A tile's rows span at most 256 * 2 * kMostLong bytes, 2.1e9.
__device__ __forceinline__ uint32_t rows_lane_off(uint32_t ld, int lane) {
    return (uint32_t)(lane >> 2) * ld * 2 + (uint32_t)(((lane & 3) ^ ((lane >> 3) & 3)) * 16);
}
// Access q of the wave.
template <int NW>
__device__ __forceinline__ void stage_rows(const f16* base, uint32_t ld, uint32_t lane_off, char* lds, int w,
                                           int q) {
    const uint32_t u = (uint32_t)(q * NW + w);
    copy_to_lds(base, lane_off, u * 32 * ld, lds + u * 1024);
}
// 32 rows (depth) of COLS fp16, for reads that transpose: the 16-byte chunk c of row r
// lies at place c ^ 2 key(r), so that the 8 rows x 32 bytes that 32 lanes read together
// (rows 0 to 3 and 8 to 11, for instance) hit different banks.
__device__ __forceinline__ int col_key(int row) { return (row & 3) | ((row >> 1) & 4); }
template <int COLS, int NW>
__device__ __forceinline__ uint32_t cols_lane_off(uint32_t ld, int lane, int w, int q) {
    constexpr int kPer = COLS / 8, kRows = 64 / kPer;   // chunks of a row; rows of an access
    const int r = lane / kPer, slot = lane % kPer;
    return (uint32_t)r * ld * 2 + (uint32_t)((slot ^ (col_key((q * NW + w) * kRows + r) << 1)) * 16);
}
template <int COLS, int NW>
__device__ __forceinline__ void stage_cols(const f16* base, uint32_t ld, uint32_t lane_off, char* lds, int w,
                                           int q) {
    constexpr int kRows = 64 / (COLS / 8);
    const uint32_t u = (uint32_t)(q * NW + w);
    copy_to_lds(base, lane_off, u * kRows * ld * 2, lds + u * 1024);
}
__device__ __forceinline__ f16x8 read_row_frag(const char* lds, int row, int chunk) {
    return *(const f16x8*)(lds + row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
}
// Fragment of 16 columns from `col`, lane l's column l % 16, depths k0 + (l / 16) * 8
// + (0..7): two transposing reads, in each of which lane t of 16 brings 4 columns of
// row t / 4 and gets column t of the 4 rows.
template <int COLS>
__device__ __forceinline__ f16x8 read_col_frag(const char* lds, int col, int k0, int lane) {
    const int t = lane & 15, row = k0 + ((lane >> 4) << 3) + (t >> 2);
    const int byte = (col + ((t & 3) << 2)) * 2;
    const char* p = lds + row * (COLS * 2) + (byte ^ (col_key(row) << 5));
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
// 16 elements of a plane; stored in one, or (plane != 0) in two that lie so far apart.
__device__ __forceinline__ void load_plane(const f16* p, f16x8* v) {
    v[0] = *(const f16x8*)p;
    v[1] = *(const f16x8*)(p + 8);
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
// 16 consecutive elements of a buffer, which may begin at any element.
__device__ __forceinline__ void load_f32(const float* p, float* v) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const f32x4 q = *(const f32x4_a4*)(p + 4 * k);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * k + e] = q[e];
    }
}
__device__ __forceinline__ void store_f32(void* to, const float* v) {
    float* p = (float*)to;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const f32x4 q = {v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]};
        *(f32x4_a4*)(p + 4 * k) = q;
    }
}
template <int DT>
__device__ __forceinline__ void store_16(void* to, const float* v) {
    uint16_t* p = (uint16_t*)to;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint16_t h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = narrow16(DT, v[8 * k + e]);
        *(u32x4_a2*)(p + 8 * k) = pack8(h);
    }
}

// acc += r l, in place: left to itself the compiler moves accumulators between registers
// in the loop (856 TFLOP/s, where these reach 1200).  It does not know that these are
// matrix instructions, whose results other instructions must not touch for some cycles:
// the accumulators are used by nothing else between the loop's first product and the
// s_nop after its last.
__device__ __forceinline__ void mul(f32x4& acc, f16x8 r, f16x8 l) {
    asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(acc) : "v"(r), "v"(l));
}

// At most N of the wave's loads into LDS are still on their way.
template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void block_sync() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

enum Kind { kGram, kSquare, kApply, kLastOrth, kLastMuon };

// What a product's kernel uses of its matrix, read once: through the table every store
// would have it read again (a tile's end took 40 us of such waits).
struct View {
    const f16 *x, *p, *q;           // X; the planes that are read
    f16 *to_x, *out;
    const float *lost_p, *lost_q;   // the planes' diagonals
    float* lost_out;
    int64_t mp, np, plane_x, plane_a;       // (the last two in elements)
    void* dst;
    int64_t offset, dst_ld;
    int32_t rows, cols, tall, dst_dtype;
    float step;                     // lr * alpha
    __device__ __forceinline__ View(const Mat& t, const Step& s, const Product& c, const MuonConsts& mc) {
        x = (const f16*)(s.ws + t.x[c.from]), to_x = (f16*)(s.ws + t.x[c.from ^ 1]);
        p = (const f16*)(s.ws + t.p[c.p]), q = (const f16*)(s.ws + t.p[c.q]);
        out = (f16*)(s.ws + t.p[c.out]);
        lost_p = (const float*)(s.ws + t.r[c.p]), lost_q = (const float*)(s.ws + t.r[c.q]);
        lost_out = (float*)(s.ws + t.r[c.out]);
        mp = t.mp, np = t.np, plane_x = t.plane_x / 2, plane_a = t.plane_a / 2;
        dst = t.dst, offset = t.offset, dst_ld = t.dst_ld;
        rows = t.rows, cols = t.cols, tall = t.tall, dst_dtype = t.dst_dtype;
        step = muon_step(t, mc);
    }
};

// The end of a tile of T x T (4 waves, a quarter each): 16 rows of 64 columns at a time,
// what the sums become and what is read for it.
template <int T, int OP, int DT, bool PRECISE>
struct Finish {
    static constexpr int FI = T / 32, FJ = T / 32;       // fragments of a wave
    static constexpr int kBlocks = FI * FJ / 4;          // of a wave
    static constexpr bool kTri = OP == kGram || OP == kSquare;
    // What a block reads: 16 elements per lane of P or X, of Q or X's lower part, of P's
    // lower part, of the weights.
    struct Beside {
        f16x8 h[2], l[2], g[2];
        float p[16];
    };
    const Product& c;
    const View& t;
    const MuonBufs& mb;
    const MuonConsts& mc;
    Item it;
    int lane, wi, wj;
    char* mine;             // 16 x kTurn floats of LDS
    float* sides;           // 2 T floats of LDS: what P's diagonal lost in the tile's rows;
                            // what Q's lost in its columns, or P's diagonal in its rows
    float step;             // lr * alpha / kScaleX

    __device__ __forceinline__ void begin() {
        step = OP == kLastMuon ? t.step * (1.0f / kScaleX) : 0.0f;
        if constexpr (OP != kGram && !PRECISE) {
            const float* p = t.lost_p + (int64_t)it.i * T;
            const float* q = OP == kSquare ? t.lost_q + (int64_t)it.j * T : p + t.mp;
            for (int e = threadIdx.x; e < T; e += 256) {
                sides[e] = p[e];
                sides[T + e] = q[e];
            }
            __syncthreads();
        }
    }
    // the lane's row and first column of block ij: of the tile's matrix, and of the
    // result in memory (with how many of 16 columns exist)
    __device__ __forceinline__ void place(int ij, int64_t& row, int64_t& col) const {
        row = (int64_t)it.i * T + wi + ij / (FJ / 4) * 16 + (lane >> 2);
        col = (int64_t)it.j * T + wj + ij % (FJ / 4) * 64 + ((lane & 3) << 4);
    }
    __device__ __forceinline__ int result_place(int ij, int64_t& r, int64_t& col) const {
        place(ij, r, col);
        if (t.tall) {
            const int64_t top = r - (lane >> 2);
            r = col - ((lane & 3) << 4) + lane;
            col = top;
        }
        return r < t.rows && col < t.cols ? (int)(t.cols - col < 16 ? t.cols - col : 16) : 0;
    }
    __device__ __forceinline__ void fetch(int ij, Beside& d) const {
        int64_t row, col;
        place(ij, row, col);
        if constexpr (OP == kSquare) {
            const int64_t at = row * t.mp + col;
            load_plane(t.p + at, d.h);
            if constexpr (PRECISE) {
                load_plane(t.p + t.plane_a + at, d.l);
            } else {
                load_plane(t.q + at, d.l);
                if (c.lower) {
                    load_plane(t.p + t.plane_a + at, d.g);
                } else {
                    d.g[0] = d.g[1] = f16x8{0, 0, 0, 0, 0, 0, 0, 0};
                }
            }
        } else if constexpr (!kTri) {
            const int64_t at = row * t.np + col;
            load_plane(t.x + at, d.h);
            load_plane(t.x + t.plane_x + at, d.l);
        }
        if constexpr (OP == kLastMuon) {
            const int n = result_place(ij, row, col);
            if (n == 16) load_f32(mb.master + t.offset + row * t.cols + col, d.p);
        }
    }
    // 16 consecutive elements of the result, of X's values v, and of the weights p
    __device__ __forceinline__ void result(int64_t r, int64_t k, float* v, const float* p) const {
        if constexpr (OP == kLastOrth) {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] *= 1.0f / kScaleX;
            char* out = (char*)t.dst + (r * t.dst_ld + k) * (t.dst_dtype == ZERO_FP32 ? 4 : 2);
            if (t.dst_dtype == ZERO_FP32) store_f32(out, v);
            else if (t.dst_dtype == ZERO_FP16) store_16<ZERO_FP16>(out, v);
            else store_16<ZERO_BF16>(out, v);
        } else if constexpr (OP == kLastMuon) {
            const int64_t e0 = t.offset + r * t.cols + k;
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = p[e] * mc.decay - step * v[e];
            store_f32(mb.master + e0, v);
            store_16<DT>(mb.p16 + e0, v);
        }
    }
    __device__ __forceinline__ void result_one(int64_t r, int64_t k, float v) const {
        if constexpr (OP == kLastOrth) {
            store_elem(t.dst, r * t.dst_ld + k, t.dst_dtype, v * (1.0f / kScaleX));
        } else if constexpr (OP == kLastMuon) {
            const int64_t e0 = t.offset + r * t.cols + k;
            const float p = mb.master[e0] * mc.decay - step * v;
            mb.master[e0] = p;
            mb.p16[e0] = narrow16(DT, p);
        }
    }
    // Lane l brings row l % 16 and 4 columns from (l / 16) * 4 of 4 fragments.
    __device__ __forceinline__ void block(int ij, const f32x4* sums, const Beside& d) const {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *(f32x4*)(mine + ((lane & 15) * kTurn + j * 16 + ((lane >> 4) << 2)) * 4) = sums[j];
        wave_sync();
        int64_t row, col;
        place(ij, row, col);
        float* at = (float*)mine + (lane >> 2) * kTurn + ((lane & 3) << 4);
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = at[e];
        if constexpr (kTri) {
            f16* out = t.out;
            const int64_t lower = PRECISE || (OP == kGram && c.lower) ? t.plane_a : 0;
            if constexpr (OP == kGram) {
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] *= c.fc;
            } else if constexpr (PRECISE) {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    v[e] = c.fp * ((float)d.h[e >> 3][e & 7] + (float)d.l[e >> 3][e & 7]) + c.fc * v[e];
            } else {
                // to first order, what the diagonals of P and Q lost
                const float lost_p = sides[row - (int64_t)it.i * T];
                const float* lost_q = sides + T + (col - (int64_t)it.j * T);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float p = (float)d.h[e >> 3][e & 7], q = (float)d.l[e >> 3][e & 7];
                    v[e] += p * lost_q[e] + lost_p * q;
                    v[e] = c.fp * (p + (float)d.g[e >> 3][e & 7]) + c.fq * q + c.fc * v[e];
                }
                if (it.i == it.j) {
                    const float own = c.lower ? 0.0f : c.fp * lost_p;
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (row == col + e) v[e] += own + c.fq * lost_q[e];
                }
            }
            // Below the diagonal as it is, above it turned over, in the diagonal's tiles too:
            // a product of planes that are not quite symmetric is not quite either, and the
            // next one, which reads rows for columns, would not be one of the same polynomial
            // (96 x 300 was off by 4e-3 in the place of 5e-4).
            const int64_t turned = col - ((lane & 3) << 4) + lane, top = row - (lane >> 2);
            if (it.i != it.j) {
                store_plane(out + row * t.mp + col, lower, v);
                turn_over(mine, at, v, lane);
                store_plane(out + turned * t.mp + top, lower, v);
            } else {
                float turned_v[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) turned_v[e] = v[e];
                turn_over(mine, at, turned_v, lane);
                // the 16 x 16 on the diagonal: above it, the element across
                const int r = lane >> 2;
                const float* across = (const float*)mine + ((lane & 3) << 4) + r;
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (col == top && e > r) v[e] = across[e * kTurn];
                if (col <= top) store_plane(out + row * t.mp + col, lower, v);
                if ((turned & ~int64_t(15)) < top) store_plane(out + turned * t.mp + top, lower, turned_v);
                if constexpr (!PRECISE) {
                    float u = 0.0f;
#pragma unroll
                    for (int e = 0; e < 16; ++e) u = e == r ? v[e] : u;
                    if (col == top) {
                        t.lost_out[row] = u - (float)(f16)u;
                        t.lost_out[t.mp + row] = u;
                    }
                }
            }
        } else {
            float lost_p = 0.0f, diag_p = 0.0f;
            if constexpr (!PRECISE) {
                lost_p = sides[row - (int64_t)it.i * T];
                diag_p = sides[T + row - (int64_t)it.i * T];
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float h = (float)d.h[e >> 3][e & 7], l = (float)d.l[e >> 3][e & 7];
                // to first order, what P's diagonal lost, and P times X's lower part
                if constexpr (!PRECISE) v[e] += lost_p * h + diag_p * l;
                v[e] = c.fp * (h + l) + c.fc * v[e];
            }
            if constexpr (OP == kApply) {
                store_plane(t.to_x + row * t.np + col, t.plane_x, v);
            } else {
                // in memory: row r, 16 consecutive columns from k, or what of them exists
                int64_t r, k;
                const int n = result_place(ij, r, k);
#pragma unroll
                for (int e = 0; e < 16; ++e) at[e] = v[e];
                wave_sync();
                const float* from = t.tall ? (const float*)mine + lane : at;
                const int every = t.tall ? kTurn : 1;
                if (n == 16) {
                    if (t.tall) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] = from[e * kTurn];
                    }
                    result(r, k, v, d.p);
                } else {
                    for (int e = 0; e < n; ++e) result_one(r, k + e, from[e * every]);
                }
            }
        }
        wave_sync();
    }
};

template <size_t... I, typename F>
__device__ __forceinline__ void each_of(std::index_sequence<I...>, F&& f) {
    (f(std::integral_constant<size_t, I>{}), ...);
}

// A tile of one product, or a part of its depth: T x T by 4 waves, a quarter each, with
// the sums in registers.  Stages of 32 of the depth go from memory into LDS three ahead of
// their products, and from LDS into registers one ahead: 75 to 77 % of the matrix cores'
// cycles in the loop (1324 TFLOP/s).
// Ends whose reads begin before the loop, and ends in loops (26 kB of code, not 58), take the
// same time: what a tile's end costs are its planes' bytes, at once from all blocks.
template <int T, int OP, int DT, bool PRECISE>
__global__ void __launch_bounds__(256, T == 256 ? 1 : 2)
matrix_product_kernel(Step s, Product c, MuonBufs mb, MuonConsts mc) {
    using End = Finish<T, OP, DT, PRECISE>;
    constexpr int NW = 4, FI = End::FI, FJ = End::FJ;
    constexpr bool kTri = End::kTri;
    constexpr int kSide = T * kBK * 2;      // bytes of a side's stage
    if (skipped(s.res)) return;
    // four arrays, so that the compiler sees that reads of one do not wait for loads
    // into another
    __shared__ __attribute__((aligned(1024))) char lds0[2 * kSide];
    __shared__ __attribute__((aligned(1024))) char lds1[2 * kSide];
    __shared__ __attribute__((aligned(1024))) char lds2[2 * kSide];
    __shared__ __attribute__((aligned(1024))) char lds3[2 * kSide];
    const int64_t cut = (int64_t)blockIdx.x - c.cut.whole;
    const int64_t n_cut = s.n_items - c.cut.whole;
    const int part = cut < 0 ? 0 : (int)(cut / n_cut), parts = cut < 0 ? 1 : c.cut.parts;
    const Item it = s.items[cut < 0 ? item_of<32>(blockIdx.x, c.cut.whole) : c.cut.whole + cut % n_cut];
    const View t(s.mats[it.mat], s, c, mc);
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wi = (w / 2) * (T / 2), wj = (w % 2) * (T / 2);
    const int64_t i0 = (int64_t)it.i * T, j0 = (int64_t)it.j * T;
    const int64_t np = t.np, mp = t.mp;
    const f16 *left, *right;
    int64_t left_plane, right_plane, left_ld, right_ld;
    int depth;
    if constexpr (OP == kGram) {
        left = t.x + i0 * np, right = t.x + j0 * np;
        left_plane = right_plane = t.plane_x, left_ld = right_ld = np, depth = (int)np;
    } else if constexpr (OP == kSquare) {
        left = t.p + i0 * mp, right = t.q + j0 * mp;
        left_plane = right_plane = t.plane_a, left_ld = right_ld = mp, depth = (int)mp;
    } else {
        left = t.p + i0 * mp, right = t.x + j0;
        left_plane = t.plane_a, right_plane = t.plane_x, left_ld = mp, right_ld = np, depth = (int)mp;
    }
    f32x4 acc[FI][FJ];
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int j = 0; j < FJ; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const uint32_t left_off = rows_lane_off((uint32_t)left_ld, lane);
    // of even and odd accesses: the key of the columns' rows has a period of 16 rows
    uint32_t right_off[2];
#pragma unroll
    for (int q = 0; q < 2; ++q)
        right_off[q] = kTri ? rows_lane_off((uint32_t)right_ld, lane)
                            : cols_lane_off<T, NW>((uint32_t)right_ld, lane, w, q);
    static_assert(NW * (512 / T) * 2 % 16 == 0, "the key's period");
    // stages of the precise form: lo hi, hi lo, hi hi, the small ones first, so that they are
    // not rounded to the bits of the large ones' sum.  A part has a share of them, in fours.
    const int per = depth / kBK, fours = (PRECISE ? 3 * per : per) / 4;
    const int first = (int)((int64_t)fours * part / parts) * 4;
    const int total = (int)((int64_t)fours * (part + 1) / parts) * 4 - first;
    const int64_t step_r = kTri ? kBK : (int64_t)kBK * right_ld;
    int seg = PRECISE ? first / per : 0;
    int left_in_seg = per - (first - seg * per);
    const f16* next_l = left + (PRECISE && seg == 0 ? left_plane : 0) + (int64_t)(first - seg * per) * kBK;
    const f16* next_r = right + (seg == 1 ? right_plane : 0) + (int64_t)(first - seg * per) * step_r;
    constexpr int kSideLoads = kSide / 1024 / NW, kLoads = 2 * kSideLoads;   // of a wave
    auto load_piece = [&](char* lds, int q) {       // access q of the next stage
        if (q < kSideLoads) stage_rows<NW>(next_l, (uint32_t)left_ld, left_off, lds, w, q);
        else if constexpr (kTri)
            stage_rows<NW>(next_r, (uint32_t)right_ld, right_off[(q - kSideLoads) & 1], lds + kSide, w,
                           q - kSideLoads);
        else
            stage_cols<T, NW>(next_r, (uint32_t)right_ld, right_off[(q - kSideLoads) & 1], lds + kSide, w,
                              q - kSideLoads);
    };
    // Past the last stage the same one is loaded again, which nothing reads.
    int left_in_all = total;
    auto loaded = [&] {
        const bool go = --left_in_all > 0;
        next_l += go ? kBK : 0;
        next_r += go ? step_r : 0;
        if constexpr (PRECISE) {
            const bool last = --left_in_seg == 0 && go;   // selected, not branched to
            left_in_seg = last ? per : left_in_seg;
            seg += last;
            next_l = last ? left : next_l;
            next_r = last ? right + (seg == 1 ? right_plane : 0) : next_r;
        }
    };
    auto load = [&](char* lds) {
#pragma unroll
        for (int q = 0; q < kLoads; ++q) load_piece(lds, q);
        loaded();
    };
    struct Frags {
        f16x8 l[FI], r[FJ];
    };
    auto read_piece = [&](Frags& f, const char* lds, int q) {
        if (q < FI) f.l[q] = read_row_frag(lds, wi + q * 16 + (lane & 15), lane >> 4);
        else if constexpr (kTri)
            f.r[q - FI] = read_row_frag(lds + kSide, wj + (q - FI) * 16 + (lane & 15), lane >> 4);
        else f.r[q - FI] = read_col_frag<T>(lds + kSide, wj + (q - FI) * 16, 0, lane);
    };
    // One stage: its products from registers, while the next stage's fragments come from
    // LDS and the stage after the next two goes into LDS, a few of each in turn.
    constexpr int kTurns = FI + FJ, kMuls = FI * FJ / kTurns, kEvery = kTurns / kLoads;
    static_assert(kMuls * kTurns == FI * FJ && kEvery * kLoads == kTurns, "even turns");
    auto phase = [&](const Frags& now, Frags& next, const char* from_lds, char* to_lds) {
#pragma unroll
        for (int q = 0; q < kTurns; ++q) {
            read_piece(next, from_lds, q);
            if (q % kEvery == 0) load_piece(to_lds, q / kEvery);
#pragma unroll
            for (int e = q * kMuls; e < (q + 1) * kMuls; ++e) mul(acc[e / FJ][e % FJ], now.r[e % FJ], now.l[e / FJ]);
            __builtin_amdgcn_sched_barrier(0);
        }
        loaded();
        // the next stage but one has to be there; what was loaded here may be on its way
        wait_loads<kLoads>();
        block_sync();
    };
    Frags f0, f1;
    load(lds0);
    load(lds1);
    load(lds2);
    wait_loads<kLoads>();
    block_sync();
#pragma unroll
    for (int q = 0; q < kTurns; ++q) read_piece(f0, lds0, q);
    int k = 0;
    do {                        // there are at least 4 stages
        phase(f0, f1, lds1, lds3);
        phase(f1, f0, lds2, lds0);
        phase(f0, f1, lds3, lds1);
        phase(f1, f0, lds0, lds2);
        k += 4;
    } while (k < total);
    // the last loads, into LDS that is used again below, and the last products' results,
    // which nothing else waits for
    asm volatile("s_waitcnt vmcnt(0)\n\ts_nop 15\n\ts_nop 15" ::: "memory");
    block_sync();

    if (parts > 1) {            // its sums as they are: matrix_join_kernel's work is the rest
        f32x4* sums = (f32x4*)(s.ws + s.sums_off) + (cut % n_cut * parts + part) * (T * T / 4) +
                      w * (FI * FJ * 64) + lane;
#pragma unroll
        for (int e = 0; e < FI * FJ; ++e) sums[e * 64] = acc[e / FJ][e % FJ];
        return;
    }
    // What a block reads comes kAhead blocks before it is used.
    constexpr int kAhead = 4;
    char* mine = w == 0 ? lds0 : w == 1 ? lds1 : w == 2 ? lds2 : lds3;
    constexpr int kMine = 16 * kTurn * 4;
    static_assert(2 * kSide >= kMine + 8 * T, "an array for each wave, and the sides");
    End end{c, t, mb, mc, it, lane, wi, wj, mine, (float*)(lds0 + kMine), 0.0f};
    end.begin();
    typename End::Beside d[kAhead];
#pragma unroll
    for (int ij = 0; ij < kAhead; ++ij) end.fetch(ij, d[ij]);
    // (a loop of this size the compiler would leave a loop, and the sums in memory)
    each_of(std::make_index_sequence<End::kBlocks>(), [&](auto at) {
        constexpr int ij = (int)decltype(at)::value;
        end.block(ij, &acc[ij / (FJ / 4)][ij % (FJ / 4) * 4], d[ij % kAhead]);
        if constexpr (ij + kAhead < End::kBlocks) end.fetch(ij + kAhead, d[ij % kAhead]);
        __builtin_amdgcn_sched_barrier(0);
    });
}

// The parts of cut tiles added up, in order: a block has one of the kBlocks blocks of 16
// rows of 64 columns of each of a tile's waves.
template <int T, int OP, int DT, bool PRECISE>
__global__ void __launch_bounds__(256)
matrix_join_kernel(Step s, Product c, MuonBufs mb, MuonConsts mc) {
    using End = Finish<T, OP, DT, PRECISE>;
    if (skipped(s.res)) return;
    __shared__ __attribute__((aligned(16))) float turn[4][16 * kTurn], sides[2 * T];
    const int64_t tile = blockIdx.x / End::kBlocks;
    const int ij = (int)(blockIdx.x % End::kBlocks);
    const Item it = s.items[c.cut.whole + tile];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const View t(s.mats[it.mat], s, c, mc);
    End end{c, t, mb, mc, it, lane, (w / 2) * (T / 2), (w % 2) * (T / 2), (char*)turn[w], sides, 0.0f};
    end.begin();
    typename End::Beside d;
    end.fetch(ij, d);
    f32x4 sum[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const f32x4* sums = (const f32x4*)(s.ws + s.sums_off) + tile * c.cut.parts * (T * T / 4) +
                        w * (End::FI * End::FJ * 64) + ij * 256 + lane;
    for (int k = 0; k < c.cut.parts; ++k, sums += T * T / 4)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] += sums[j * 64];
    end.block(ij, sum, d);
}

// ------------------------------------------------------------ small --------
// Matrices whose shorter side is at most 64 (a low-rank adapter's factors, vectors) go
// another way: the Gram matrix A = U U^T of the whole update, all steps on it alone,
//     Q = a + b A + c A A,   P <- Q P,   A <- Q A Q,
// and the result P U / (||U|| + eps): two passes over the matrix and three launches, all to
// 32 bits.  A's rounding grows with the square of what the steps multiply small singular
// values by, so A, Q and P are fp64.  (The way of the larger ones, three launches for
// each step, took 250 us for 56 factors of 16 x 2048, this one 40.)
constexpr int kSmall = 64;                 // shorter side, at most
constexpr int kSmallCols = 128;            // columns of the wide form that are in LDS at once
constexpr int kSmallParts = 256;           // blocks of a matrix, at most
constexpr int kSmallLd = kSmall + 4, kSmallRow = kSmallCols + 4;

// 8 elements of the update at once: item q of a chunk of kSmallCols columns from c0, as
// (i, k) of the wide form and their direction.  False past the chunk.
__device__ __forceinline__ bool small_item(const Mat& t, int q, int64_t c0, int& i, int& k, int& n) {
    if (t.tall) {
        const int per = (t.m + 7) / 8;
        k = q / per, i = q % per * 8;
        n = c0 + k < t.n ? (t.m - i < 8 ? t.m - i : 8) : 0;
        return k < kSmallCols;
    }
    i = q / (kSmallCols / 8), k = q % (kSmallCols / 8) * 8;
    const int64_t left = t.n - c0 - k;
    n = left < 0 ? 0 : left < 8 ? (int)left : 8;
    return i < t.m;
}
// A chunk of the update into LDS: by column (to[k * LD + i]), or by row (to[i * LD + k]),
// times `by0` times `by1`.
template <bool FIRST, bool BY_COLUMN, typename Source>
__device__ __forceinline__ void small_load(const Mat& t, const Source& src, int64_t c0, float by0, float by1,
                                           float* to) {
    for (int q = threadIdx.x;; q += kThreads) {
        int i, k, n;
        if (!small_item(t, q, c0, i, k, n)) break;
        float v[8];
        if (n > 0) {
            src.template get<FIRST>(t, t.tall ? c0 + k : i, t.tall ? i : c0 + k, n, v);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int ii = t.tall ? i + e : i, kk = t.tall ? k : k + e;
            if (ii < kSmall) to[BY_COLUMN ? kk * kSmallLd + ii : ii * kSmallRow + kk] = v[e] * by0 * by1;
        }
    }
}

// First pass: a block's part of U U^T, its columns' sums in fp64.  A thread has 4 x 4
// elements of A and every S-th column.
template <typename Source>
__global__ void __launch_bounds__(kThreads)
small_gram_kernel(Step s, Source src) {
    if (skipped(s.res)) return;
    src.begin(s);
    __shared__ __attribute__((aligned(16))) float u[kSmallCols * kSmallLd];
    __shared__ double red[16][kThreads];
    const Item it = s.items[blockIdx.x];
    const Mat t = s.mats[it.mat];
    const int side = (t.m + 3) / 4, blocks = side * side, slices = kThreads / blocks;
    const int blk = (int)threadIdx.x % blocks, slice = (int)threadIdx.x / blocks;
    const int bi = blk / side * 4, bj = blk % side * 4;
    for (int e = threadIdx.x; e < kSmallCols * kSmallLd; e += kThreads) u[e] = 0.0f;
    __syncthreads();
    double acc[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = 0.0;
    const int64_t end = (int64_t)(it.i + 1) * t.np < t.n ? (int64_t)(it.i + 1) * t.np : t.n;
    for (int64_t c0 = (int64_t)it.i * t.np; c0 < end; c0 += kSmallCols) {
        small_load<true, true>(t, src, c0, 1.0f, 1.0f, u);
        __syncthreads();
        if (slice < slices) {
            for (int k = slice; k < kSmallCols; k += slices) {
                const f32x4 x = *(const f32x4*)(u + k * kSmallLd + bi), y = *(const f32x4*)(u + k * kSmallLd + bj);
#pragma unroll
                for (int p = 0; p < 4; ++p)
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[p * 4 + q] = fma((double)x[p], (double)y[q], acc[p * 4 + q]);
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) red[e][threadIdx.x] = acc[e];
    __syncthreads();
    double* out = (double*)(s.ws + t.p[0]) + (int64_t)it.i * blocks * 16;
    for (int e = threadIdx.x; e < blocks * 16; e += kThreads) {
        double sum = 0.0;
        for (int k = 0; k < slices; ++k) sum += red[e & 15][k * blocks + (e >> 4)];
        out[e] = sum;
    }
}

// One block per matrix: A from its parts, and the steps.
struct SmallNs {
    double a, b, c, eps;
    int32_t steps, pad;
};
// A thread has R x R elements of all products: of 16 x 2048 matrices (R = 1) the launch took
// 31 us where 16 threads had 4 x 4 each, and 9.7 with an element for each of 256.
constexpr int kStepsLd = kSmall + 1;
template <int R>
__device__ __forceinline__ void small_steps(const Step& s, const SmallNs& ns, const Mat& t, double* A, double* Q,
                                            double* P, double* W, double* norm) {
    constexpr int kSide = 16 * R, kLd = kStepsLd;
    const int side = (t.m + 3) / 4, blocks = side * side, tid = threadIdx.x;
    const int bi = tid / 16 * R, bj = tid % 16 * R;
    const double* part = (const double*)(s.ws + t.p[0]);
    for (int e = tid; e < kSide * kLd; e += kThreads) A[e] = 0.0;
    __syncthreads();
    for (int e = tid; e < blocks * 16; e += kThreads) {
        double sum = 0.0;
#pragma unroll 8
        for (int k = 0; k < t.n_parts; ++k) sum += part[(int64_t)k * blocks * 16 + e];
        const int b = e >> 4, p = (e & 15) >> 2, q = e & 3;
        A[(b / side * 4 + p) * kLd + b % side * 4 + q] = sum;
    }
    __syncthreads();
    if (tid == 0) {
        double sum = 0.0;
        for (int k = 0; k < t.m; ++k) sum += A[k * kLd + k];
        *norm = sqrt(sum) + ns.eps;
        store_factor((float*)(s.ws + t.r[0]), 1.0 / *norm);
    }
    __syncthreads();
    double c[R * R];
    auto product = [&](const double* x, const double* y) {     // the thread's part of x y
#pragma unroll
        for (int e = 0; e < R * R; ++e) c[e] = 0.0;
#pragma unroll(R == 1 ? 16 : 4)
        for (int k = 0; k < kSide; ++k) {
            double u[R], v[R];
#pragma unroll
            for (int p = 0; p < R; ++p) u[p] = x[(bi + p) * kLd + k], v[p] = y[k * kLd + bj + p];
#pragma unroll
            for (int e = 0; e < R * R; ++e) c[e] = fma(u[e / R], v[e % R], c[e]);
        }
        __syncthreads();
    };
    auto each = [&](auto&& f) {                                 // f(element, its product)
#pragma unroll
        for (int e = 0; e < R * R; ++e) f((bi + e / R) * kLd + bj + e % R, c[e], bi + e / R == bj + e % R);
        __syncthreads();
    };
    const double inv = 1.0 / (*norm * *norm);
    each([&](int at, double, bool) { A[at] *= inv; });
    for (int k = 0; k < ns.steps; ++k) {
        product(A, A);
        each([&](int at, double v, bool diag) {
            Q[at] = (diag ? ns.a : 0.0) + ns.b * A[at] + ns.c * v;
            if (k == 0) P[at] = Q[at];
        });
        if (k > 0) {
            product(Q, P);
            each([&](int at, double v, bool) { P[at] = v; });
        }
        if (k + 1 == ns.steps) break;
        product(Q, A);
        each([&](int at, double v, bool) { W[at] = v; });
        product(W, Q);
        each([&](int at, double v, bool) { A[at] = v; });
    }
    float* out = (float*)(s.ws + t.p[1]);
    for (int e = tid; e < side * 4 * kSmall; e += kThreads) {
        const int i = e / kSmall, j = e % kSmall;
        out[e] = j < side * 4 ? (float)P[i * kLd + j] : 0.0f;
    }
}
__global__ void __launch_bounds__(kThreads)
small_steps_kernel(Step s, SmallNs ns) {
    if (skipped(s.res)) return;
    __shared__ double A[kSmall * kStepsLd], Q[kSmall * kStepsLd], P[kSmall * kStepsLd], W[kSmall * kStepsLd];
    __shared__ double norm;
    const Mat t = s.mats[blockIdx.x];
    if (t.m <= 16) small_steps<1>(s, ns, t, A, Q, P, W, &norm);
    else if (t.m <= 32) small_steps<2>(s, ns, t, A, Q, P, W, &norm);
    else small_steps<4>(s, ns, t, A, Q, P, W, &norm);
}

// Second pass: P (U / norm), a block's columns, and what becomes of it.  A thread has 4 rows
// and 4 columns at a time.
template <bool MUON, int DT, typename Source>
__global__ void __launch_bounds__(kThreads)
small_apply_kernel(Step s, Source src, MuonBufs mb, MuonConsts mc) {
    if (skipped(s.res)) return;
    src.begin(s);
    __shared__ __attribute__((aligned(16))) float u[kSmall * kSmallRow];
    __shared__ __attribute__((aligned(16))) float P[kSmall * kSmall];
    const Item it = s.items[blockIdx.x];
    const Mat t = s.mats[it.mat];
    const int side = (t.m + 3) / 4;
    const float inv[2] = {((const float*)(s.ws + t.r[0]))[0], ((const float*)(s.ws + t.r[0]))[1]};
    for (int e = threadIdx.x; e < side * 4 * kSmall; e += kThreads) P[e] = ((const float*)(s.ws + t.p[1]))[e];
    for (int e = threadIdx.x; e < kSmall * kSmallRow; e += kThreads) u[e] = 0.0f;
    __syncthreads();
    const float step = MUON ? muon_step(t, mc) : 0.0f;
    const int64_t end = (int64_t)(it.i + 1) * t.np < t.n ? (int64_t)(it.i + 1) * t.np : t.n;
    for (int64_t c0 = (int64_t)it.i * t.np; c0 < end; c0 += kSmallCols) {
        small_load<false, false>(t, src, c0, inv[0], inv[1], u);
        __syncthreads();
        for (int q = threadIdx.x; q < side * (kSmallCols / 4); q += kThreads) {
            const int i = q / (kSmallCols / 4) * 4, k = q % (kSmallCols / 4) * 4;
            float o[4][4] = {{0, 0, 0, 0}, {0, 0, 0, 0}, {0, 0, 0, 0}, {0, 0, 0, 0}};
            for (int j = 0; j < t.m; ++j) {
                const f32x4 x = *(const f32x4*)(P + j * kSmall + i), y = *(const f32x4*)(u + j * kSmallRow + k);
#pragma unroll
                for (int a = 0; a < 4; ++a)
#pragma unroll
                    for (int b = 0; b < 4; ++b) o[a][b] = fmaf(x[a], y[b], o[a][b]);
            }
            // four runs of up to 4 elements in memory
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const int64_t r = t.tall ? c0 + k + a : i + a, c = t.tall ? i : c0 + k;
                if (r >= t.rows) continue;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    if (c + b >= t.cols) continue;
                    const float v = t.tall ? o[b][a] : o[a][b];
                    if constexpr (MUON) {
                        const int64_t at = t.offset + r * t.cols + c + b;
                        const float w = mb.master[at] * mc.decay - step * v;
                        mb.master[at] = w;
                        mb.p16[at] = narrow16(DT, w);
                    } else {
                        store_elem(t.dst, r * t.dst_ld + c + b, t.dst_dtype, v);
                    }
                }
            }
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------ host ---------
int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// The tile of a matrix's products, by its shorter side.
// 256 wide ones do up to 1.7 times the work of 128 wide ones in the same time, which need
// more of LDS than of the matrix cores; these are more, and each shorter.  Shorter sides of up
// to kTogether take 256 wide ones where the list has `many` of them, on and below the diagonals:
// 36 of 1024 x 1024 (360) take 1645 us with 128 and 1754 with 256, 42 (420) 1866 and 1850, 48
// (480) 2097 and 1934.  In 32 bits 12 (120) 1206 and 1344, 15 (150) 1491 and 1438, 18 (180) 1978
// and 1759; 60 of 500 x 500 (180) 1037 and 1049, 120 (360) 2301 and 2101.  Where 256 pads more
// than 128 does it never pays: 120 of 600 x 600 1766 and 2523, 100 of 800 x 800 3112 and 3759.
constexpr int64_t kTogether = 1024, kMany = 420, kManyPrecise = 180;
int tile_for(int64_t m, bool many) {
    return m > kTogether || (many && up(m, 256) == up(m, 128)) ? 256 : 128;
}
// Whether two steps go together: with Q = a + B, the second step's A is Q A Q and what
// both do to X is Q' Q, 5 products of m x m (half computed) in the place of 2 and of one
// of m x n by its transpose and one of m x m by m x n: fewer operations where n > m.  The
// planes' roundings then go through four products and not two, and weigh 2 to 5 times as much
// in a matrix of low rank, the more the smaller it is: 65 x 200 of rank 16 is off by 6.0e-3 in
// pairs, 1040 x 2800 of rank 65 by 2.7e-3, 2048 x 4096 of rank 128 by 1.6e-3.
constexpr int64_t kLeastPairs = 2048;
bool pairs_for(int64_t m, int64_t n) { return m >= kLeastPairs && 2 * n >= 3 * m; }
// A list of so few 128 wide tiles below the diagonals goes through the steps together, with
// 128 wide tiles (and in pairs where pairs_for says so of all): one matrix of 2048 x 2048 (136
// tiles) in 390 us and not 525, of 2816 x 2816 (253) in 699 and not 837, two of 2048 x 2048
// (272) in 685 and not 739, but one of 3000 x 3000 (300) in 1059 and not 942, two of 2304 x
// 2304 (342) in 858 and not 822.  In 32 bits one of 1500 x 1500 (78) takes 558 us and not 579,
// one of 1664 x 5504 (91) 1290 and not 1236, of 2048 x 5504 (136) 1846 and not 1506.  Where the
// list would be several groups, one after the other, and is one round of blocks together, too: 3
// of 1500 x 1700 and 9 of 800 x 900 in 717 us and not 1051, in 32 bits in 1688 and not 2010.
constexpr int64_t kFew = 272, kFewPrecise = 80, kRound = 512;
// Tiles below the diagonal of a group of matrices, and bytes of its planes, after
// which the next matrix begins another group.
constexpr int64_t kGroupTiles = 1024, kGroupBytes = int64_t(4) << 30;

// How the tiles of a product are cut: the last n % slots of them are the last round of
// blocks on the device.  Costs are in stages of a tile: a block's begin and end, and what
// the parts' sums (64 kB or 256 kB each) and the second launch take.  Without these, two of
// 2048 x 2048 took 1084 us in the place of 745, one 666 in the place of 535.
Cut cut_for(int64_t n, int tile, int64_t stages) {
    const int64_t slots = tile == 256 ? 256 : 512, rest = n % slots;
    Cut best = {n, 1, 0};
    if (rest == 0) return best;
    const int64_t ends = 2048 / tile;
    int64_t least = stages + ends;
    for (int64_t parts = 2; parts <= 16 && parts * rest <= 2 * slots && stages / parts >= 8; ++parts) {
        const int64_t rounds = (parts * rest + slots - 1) / slots;
        const int64_t cost = rounds * ((stages + parts - 1) / parts + ends) + parts * rest / ends + 3 * ends / 2;
        if (cost < least) {
            least = cost;
            best = {n - rest, (int32_t)parts, 0};
        }
    }
    return best;
}

// Columns whose products are added up in one chain of fp32 sums, 1024 of 32 products each: of
// a longer matrix, which is a group of its own, every tile of A is cut, in 32 bits into three
// times as many parts.  In 16 chains at most 70 x 4000000 was off by 9.1e-6 in 32 bits and not
// 1.2e-6, with all entries alike by 1.8e-3 and not 3e-5.
constexpr int64_t kMostDepth = 32768;

struct Build {
    std::vector<Group> groups;
    std::vector<Mat> mats;
    std::vector<Item> items;
    int64_t ws = 0;

    bool add(const Mat* in, int64_t count, int tile, bool pairs, bool precise) {
        // longest products first: the last round of blocks is then a short one
        std::vector<Mat> v(in, in + count);
        std::stable_sort(v.begin(), v.end(), [](const Mat& x, const Mat& y) { return x.np > y.np; });
        Group g;
        memset(&g, 0, sizeof g);
        g.tile = tile, g.pairs = pairs;
        g.mat0 = (int64_t)mats.size(), g.n_mats = count;
        int64_t at = 0, parts = 0;
        const int planes = precise ? 2 : 1;
        for (Mat& t : v) {
            t.plane_x = (int64_t)t.mp * t.np * 2, t.plane_a = (int64_t)t.mp * t.mp * 2;
            t.x[0] = at, at = up(at + 2 * t.plane_x, 256);
            t.x[1] = at, at = up(at + 2 * t.plane_x, 256);
            for (int k = 0; k < (pairs ? 3 : 2); ++k) {
                // pairs: A has its lower part, in its own terms
                t.p[k] = at, at = up(at + (pairs && k == 0 ? 2 : planes) * t.plane_a, 256);
                t.r[k] = at, at = up(at + 8 * t.mp, 256);
            }
            const int64_t u = up(t.mp, kUnitM) / kUnitM * (up(t.np, kUnitN) / kUnitN);
            if (u > INT32_MAX) return false;
            t.part0 = parts, t.n_parts = (int32_t)u;
            parts += u;
        }
        g.inv_off = at, at = up(at + 8 * count, 256);
        g.part_off = at, at = up(at + 8 * parts, 256);
        g.sums_off = at;
        g.unit0 = (int64_t)items.size();
        for (int64_t k = 0; k < count; ++k)
            for (int64_t i = 0; i * kUnitM < v[k].mp; ++i)
                for (int64_t j = 0; j * kUnitN < v[k].np; ++j) item(g.mat0 + k, i, j);
        g.n_units = (int64_t)items.size() - g.unit0;
        // blocks of 8 x 8 tiles (below the diagonal), and bands of 4 rows in each column
        // by column: 32 consecutive tiles, an XCD's, share rows and columns
        g.tri0 = (int64_t)items.size();
        for (int64_t k = 0; k < count; ++k) {
            const int64_t q = v[k].mp / tile;
            for (int64_t bi = 0; bi < q; bi += 8)
                for (int64_t bj = 0; bj <= bi; bj += 8)
                    for (int64_t i0 = bi; i0 < bi + 8 && i0 < q; i0 += 4)
                        for (int64_t j = bj; j < bj + 8 && j < q; ++j)
                            for (int64_t i = std::max(i0, j); i < i0 + 4 && i < q; ++i) item(g.mat0 + k, i, j);
        }
        g.n_tri = (int64_t)items.size() - g.tri0;
        g.full0 = (int64_t)items.size();
        for (int64_t k = 0; k < count; ++k)
            for (int64_t i = 0; i * tile < v[k].mp; i += 4)
                for (int64_t j = 0; j * tile < v[k].np; ++j)
                    for (int64_t q = i; q < i + 4 && q * tile < v[k].mp; ++q) item(g.mat0 + k, q, j);
        g.n_full = (int64_t)items.size() - g.full0;
        int64_t short_n = INT64_MAX, short_m = INT64_MAX;
        for (const Mat& t : v) {
            short_n = std::min<int64_t>(short_n, t.np);
            short_m = std::min<int64_t>(short_m, t.mp);
        }
        const int64_t thrice = precise ? 3 : 1;
        g.gram = cut_for(g.n_tri, tile, thrice * short_n / kBK);
        if (short_n > kMostDepth) {
            const int64_t parts = thrice * ((short_n + kMostDepth - 1) / kMostDepth);
            g.gram = {0, (int32_t)std::max<int64_t>(parts, g.gram.whole == 0 ? g.gram.parts : 1), 0};
        }
        g.square = cut_for(g.n_tri, tile, thrice * short_m / kBK);
        g.apply = cut_for(g.n_full, tile, thrice * short_m / kBK);
        int64_t sums = 0;
        for (const auto& c : {std::make_pair(g.gram, g.n_tri), std::make_pair(g.square, g.n_tri),
                              std::make_pair(g.apply, g.n_full)})
            if (c.first.parts > 1) sums = std::max(sums, (c.second - c.first.whole) * c.first.parts);
        ws = std::max(ws, up(at + sums * tile * tile * 4, 256));
        if (g.n_units > kMaxLaunchBlocks || g.n_full > kMaxLaunchBlocks ||
            (g.n_tri - g.gram.whole) * g.gram.parts > kMaxLaunchBlocks)
            return false;
        mats.insert(mats.end(), v.begin(), v.end());
        groups.push_back(g);
        return true;
    }
    // Matrices with a shorter side of at most kSmall, all at once.
    bool add_small(const std::vector<Mat>& in) {
        Group g;
        memset(&g, 0, sizeof g);
        g.mat0 = (int64_t)mats.size(), g.n_mats = (int64_t)in.size();
        g.unit0 = (int64_t)items.size();
        int64_t at = 0;
        for (Mat t : in) {
            const int64_t chunks = (t.n + kSmallCols - 1) / kSmallCols;
            const int64_t per = (chunks + kSmallParts - 1) / kSmallParts;     // of a block
            const int64_t side = (t.m + 3) / 4;
            t.np = (int32_t)(per * kSmallCols);
            t.n_parts = (int32_t)((chunks + per - 1) / per);
            t.p[0] = at, at = up(at + t.n_parts * side * side * 128, 256);
            t.p[1] = at, at = up(at + side * 4 * kSmall * 4, 256);
            t.r[0] = at, at = up(at + 8, 256);
            for (int64_t k = 0; k < t.n_parts; ++k) item((int64_t)mats.size(), k, 0);
            mats.push_back(t);
        }
        g.n_units = (int64_t)items.size() - g.unit0;
        ws = std::max(ws, at);
        groups.push_back(g);
        return g.n_units <= kMaxLaunchBlocks;
    }
    void item(int64_t mat, int64_t i, int64_t j) {
        items.push_back(Item{(uint32_t)mat, (uint16_t)i, (uint16_t)j});
    }
    int make(std::vector<Mat>& in, bool precise) {
        for (Mat& t : in) {
            t.tall = t.rows > t.cols;
            t.m = std::min(t.rows, t.cols), t.n = std::max(t.rows, t.cols);
        }
        int64_t tiles = 0;
        for (const Mat& t : in) {
            const int64_t q = up(t.m, 256) / 256;
            if (t.m > kSmall && t.m <= kTogether) tiles += q * (q + 1) / 2;
        }
        const bool many = tiles >= (precise ? kManyPrecise : kMany);
        // whether all of them go together
        int64_t tiles128 = 0;
        bool kinds[4] = {false, false, false, false}, pairs = !precise;
        for (const Mat& t : in) {
            if (t.m <= kSmall) continue;
            const int64_t q = up(t.m, 128) / 128;
            tiles128 += q * (q + 1) / 2;
            kinds[2 * (tile_for(t.m, many) == 256) + (!precise && pairs_for(t.m, t.n))] = true;
            pairs = pairs && pairs_for(t.m, t.n);
        }
        const bool one = tiles128 <= (precise ? kFewPrecise : kFew) ||
                         (tiles128 <= kRound && kinds[0] + kinds[1] + kinds[2] + kinds[3] > 1);
        auto kind_of = [&](const Mat& t) {
            return one ? (int)pairs : 2 * (tile_for(t.m, many) == 256) + (!precise && pairs_for(t.m, t.n));
        };
        std::vector<Mat> few;
        for (const Mat& t : in)
            if (t.m > 0 && t.m <= kSmall) few.push_back(t);
        if (!few.empty() && !add_small(few)) return ZERO_ERANGE;
        for (const int kind : {0, 1, 2, 3}) {
            const int tile = kind < 2 ? 128 : 256;
            const bool pairs = kind & 1;
            std::vector<Mat> v;
            int64_t tiles = 0, bytes = 0;
            for (Mat& t : in) {
                if (t.m <= kSmall || kind_of(t) != kind) continue;
                t.mp = (int32_t)up(t.m, tile), t.np = (int32_t)up(t.n, tile);
                const int64_t q = t.mp / tile;
                if (t.np > kMostDepth) {
                    if (!add(&t, 1, tile, pairs, precise)) return ZERO_ERANGE;
                    continue;
                }
                v.push_back(t);
                tiles += q * (q + 1) / 2;
                bytes += 8 * (int64_t)t.mp * t.np + 8 * (int64_t)t.mp * t.mp;
                if (tiles >= kGroupTiles || bytes >= kGroupBytes) {
                    if (!add(v.data(), (int64_t)v.size(), tile, pairs, precise)) return ZERO_ERANGE;
                    v.clear();
                    tiles = bytes = 0;
                }
            }
            if (!v.empty() && !add(v.data(), (int64_t)v.size(), tile, pairs, precise)) return ZERO_ERANGE;
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
// interleave without sharing any; a span of one row has whatever pitch the other has.
bool share(const Span& x, const Span& y) {
    if (x.end <= y.at || y.end <= x.at) return false;
    const bool one_x = x.end - x.at == x.row, one_y = y.end - y.at == y.row;
    if (x.pitch != y.pitch && !one_x && !one_y) return true;
    const uintptr_t pitch = one_x ? y.pitch : x.pitch;
    const Span &lo = x.at <= y.at ? x : y, &hi = x.at <= y.at ? y : x;
    const uintptr_t d = (hi.at - lo.at) % pitch;
    return d < lo.row || d + hi.row > pitch;
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

// Coefficients, and the powers of two that B and T (what two steps together do to X, but
// for a^2) are kept times.
struct NsConsts {
    double a, b, c;
    float eps;
    double scale_b, scale_t;
};

// Bounds of the singular values through the steps, from 1: the largest value that the
// polynomial takes between 0 and the last bound, at the end or where its derivative, a
// quadratic of x^2, is 0; of B's eigenvalues likewise; and of T's, what the polynomial applied
// twice multiplies a value by, less a^2, at 192 points (scale_for leaves a tenth to spare).
// All of them at 4096 points took 60 us of each call, more than the kernels of small lists.
bool ns_bounds(const zero_newton_schulz& ns, double* most_b, double* most_t) {
    const double a = ns.a, b = ns.b, c = ns.c;
    const double disc = 9 * b * b - 20 * a * c;
    const double half = disc >= 0 ? -0.5 * (3 * b + copysign(sqrt(disc), b)) : 0.0;
    // x^2 where the value, the slope and B's eigenvalue may have their extremes; what is not
    // inside (inf and NaN of a zero divisor among it) is passed over
    const double of_value[2] = {half / (5 * c), a / half}, of_slope = -0.3 * b / c, of_b = -0.5 * b / c;
    double r = 1.0, top_b = 0.0, top_t = 0.0, grow = 1.0;
    for (int k = 0; k < ns.steps; ++k) {
        const double end = r * r;
        auto value = [&](double l) { return fabs(sqrt(l) * (a + b * l + c * l * l)); };
        auto slope_at = [&](double l) { return fabs(a + 3 * b * l + 5 * c * l * l); };
        auto inside = [&](double l) { return l > 0 && l < end; };
        double top = value(end), slope = std::max(fabs(a), slope_at(end));
        for (const double l : of_value)
            if (inside(l)) top = std::max(top, value(l));
        if (inside(of_slope)) slope = std::max(slope, slope_at(of_slope));
        top_b = std::max(top_b, fabs(b * end + c * end * end));
        if (inside(of_b)) top_b = std::max(top_b, fabs(b * of_b + c * of_b * of_b));
        const int n = 192;
        for (int q = 1; q <= n; ++q) {
            const double x = r * q / n, l = x * x, f = a + b * l + c * l * l, ll = f * x * f * x;
            top_t = std::max(top_t, fabs((a + b * ll + c * ll * ll) * f - a * a));
        }
        grow *= slope;
        if (!(top <= kMostSigma)) return false;
        r = std::max(top, 1e-3);
    }
    *most_b = top_b, *most_t = top_t;
    return grow <= kMostGrowth;
}

// The power of two that takes values up to `most` to at most 2^15, with a tenth to spare.
bool scale_for(double most, double* scale) {
    int e = 0;
    frexp(most * 1.1 + 1e-3, &e);
    if (e > 15) return false;
    *scale = ldexp(1.0, std::min(15 - e, 14));
    return true;
}

int ns_consts(const zero_newton_schulz* ns, NsConsts* out) {
    if (!ns || ns->steps < 1 || ns->steps > 32) return ZERO_EINVAL;
    if (!isfinite(ns->a) || !isfinite(ns->b) || !isfinite(ns->c) || !isfinite(ns->eps) ||
        !(ns->eps >= 1e-30f))
        return ZERO_EINVAL;
    double most_b = 0.0, most_t = 0.0;
    if (!ns_bounds(*ns, &most_b, &most_t)) return ZERO_EINVAL;
    out->a = ns->a, out->b = ns->b, out->c = ns->c, out->eps = ns->eps;
    return scale_for(most_b, &out->scale_b) && scale_for(most_t, &out->scale_t) ? ZERO_OK : ZERO_EINVAL;
}

template <int T, int OP, int DT, bool P>
int run_product(Step s, const Item* items, int64_t n, const Cut& cut, Product c, const MuonBufs& mb,
                const MuonConsts& mc, hipStream_t stream) {
    s.items = items, s.n_items = n;
    c.cut = cut;
    int rc = launch(matrix_product_kernel<T, OP, DT, P>, cut.whole + (n - cut.whole) * cut.parts, 0, stream, s, c,
                    mb, mc);
    if (rc == ZERO_OK && cut.parts > 1)
        rc = launch(matrix_join_kernel<T, OP, DT, P>, (n - cut.whole) * Finish<T, OP, DT, P>::kBlocks, 0, stream,
                    s, c, mb, mc);
    return rc;
}

template <int T, int DT, bool P>
int run_steps(const Step& s, const Group& g, const Item* items, const NsConsts& ns, int steps, bool muon,
              const MuonBufs& mb, const MuonConsts& mc, hipStream_t stream) {
    const double a = ns.a, b = ns.b, c = ns.c, sx = kScaleX, sa = kScaleA, sb = ns.scale_b, st = ns.scale_t;
    int from = 0;
    auto square = [&](int p, int q, int out, int lower, double fp, double fq, double fc) {
        const Product d = {from, p, q, out, lower, (float)fp, (float)fq, (float)fc, {}};
        return run_product<T, kSquare, 0, P>(s, items + g.tri0, g.n_tri, g.square, d, mb, mc, stream);
    };
    for (int k = 0; k < steps;) {
        const bool two = g.pairs && k + 2 <= steps;
        const Product gram = {from, 0, 0, 0, two, 0.0f, 0.0f, (float)(sa / (sx * sx)), {}};
        int rc = run_product<T, kGram, 0, P>(s, items + g.tri0, g.n_tri, g.gram, gram, mb, mc, stream);
        // plane 0: A; plane 1: B = b A + c A A
        if (rc == ZERO_OK) rc = square(0, 0, 1, two, b * sb / sa, 0.0, c * sb / (sa * sa));
        Product last = {from, 1, 0, 0, 0, (float)a, 0.0f, (float)(1.0 / sb), {}};
        if (two) {
            // plane 2: Y = A Q = a A + A B;  plane 0: A' = Y Q = a Y + Y B
            if (rc == ZERO_OK) rc = square(0, 1, 2, 1, a, 0.0, 1.0 / sb);
            if (rc == ZERO_OK) rc = square(2, 1, 0, 0, a, 0.0, 1.0 / sb);
            // plane 2: B' = b A' + c A' A';  plane 0: T = Q' Q - a^2 = a B + a B' + B B'
            if (rc == ZERO_OK) rc = square(0, 0, 2, 0, b * sb / sa, 0.0, c * sb / (sa * sa));
            if (rc == ZERO_OK) rc = square(1, 2, 0, 0, a * st / sb, a * st / sb, st / (sb * sb));
            last = {from, 0, 0, 0, 0, (float)(a * a), 0.0f, (float)(1.0 / st), {}};
        }
        k += two ? 2 : 1;
        if (rc == ZERO_OK)
            rc = k < steps ? run_product<T, kApply, 0, P>(s, items + g.full0, g.n_full, g.apply, last, mb, mc, stream)
               : muon ? run_product<T, kLastMuon, DT, P>(s, items + g.full0, g.n_full, g.apply, last, mb, mc, stream)
                      : run_product<T, kLastOrth, 0, P>(s, items + g.full0, g.n_full, g.apply, last, mb, mc, stream);
        if (rc != ZERO_OK) return rc;
        from ^= 1;
    }
    return ZERO_OK;
}

template <int T, int DT>
int run_tiles(const Step& s, const Group& g, const Item* items, const NsConsts& ns, int steps, int precise,
              bool muon, const MuonBufs& mb, const MuonConsts& mc, hipStream_t stream) {
    return precise ? run_steps<T, DT, true>(s, g, items, ns, steps, muon, mb, mc, stream)
                   : run_steps<T, DT, false>(s, g, items, ns, steps, muon, mb, mc, stream);
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
        s.inv_off = g.inv_off, s.part_off = g.part_off, s.sums_off = g.sums_off;
        if (g.tile == 0) {
            const SmallNs small = {ns.a, ns.b, ns.c, ns.eps, steps, 0};
            Step one = s;
            one.mats = s.mats + g.mat0;
            int rc = launch(small_gram_kernel<Source>, g.n_units, 0, stream, s, src);
            if (rc == ZERO_OK) rc = launch(small_steps_kernel, g.n_mats, 0, stream, one, small);
            if (rc == ZERO_OK)
                rc = muon ? launch(small_apply_kernel<true, DT, Source>, g.n_units, 0, stream, s, src, mb, mc)
                          : launch(small_apply_kernel<false, DT, Source>, g.n_units, 0, stream, s, src, mb, mc);
            if (rc != ZERO_OK) return rc;
            continue;
        }
        int rc = launch(matrix_norm_kernel<Source>, g.n_units, 0, stream, s, src);
        if (rc != ZERO_OK) return rc;
        Step f = s;
        f.mats = s.mats + g.mat0;
        rc = launch(matrix_factor_kernel, g.n_mats, 0, stream, f, ns.eps);
        if (rc != ZERO_OK) return rc;
        rc = launch(matrix_init_kernel<Source>, g.n_units, 0, stream, s, g.mat0, src);
        if (rc != ZERO_OK) return rc;
        rc = g.tile == 128 ? run_tiles<128, DT>(s, g, items, ns, steps, precise, muon, mb, mc, stream)
                           : run_tiles<256, DT>(s, g, items, ns, steps, precise, muon, mb, mc, stream);
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
