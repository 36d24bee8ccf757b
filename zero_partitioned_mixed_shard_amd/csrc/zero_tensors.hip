// zero_tensors.hip -- operators over a table of gradient tensors (the
// zero_tensor_* calls of include/zero_shard.h): the norm of all of them and of
// each, clipping by it, and accumulation of one table into another.
//
// A plan cuts every tensor into pieces and the device table holds a record per
// piece (built there from a short list of the tensors), so a wave or block learns
// all about its work from one scalar load (no search from a block number to a
// tensor) and nothing spans two tensors: a piece's partial belongs to one
// tensor, and a tensor's norm is the sum of its pieces'.
//
// Every kernel is a streaming pass bound by HBM (at most 4 operations per
// element).  Tensors start at any element, so lanes use 16-byte (or 8-byte)
// accesses that are aligned to the element only, which gfx950 global memory
// takes as they are; pieces are cut so that all but a tensor's first begin at a
// multiple of 128 bytes of its output, and the norm, whose rate suffers, shifts
// 16-bit data that begins between dwords (run_norm).
//
// Numerics: the squares and their sums are fp64 (the square of an fp32 value
// is exact there, and the sum cannot overflow), the unscale factor is applied
// to the sum; products and sums of the other calls are fp32, rounded to the
// output's type once.  Sums are folded in a fixed order, which for the norm goes
// by the tensors' numbers of elements alone.

#include <math.h>
#include <string.h>

#include <algorithm>
#include <new>
#include <vector>

#include "zero_common.h"

namespace {

// One piece in the device table.  The outputs' addresses are an array of their
// own after the pieces.
struct Piece {
    const void* src;
    int32_t tensor;    // index in the table
    uint32_t info;     // elements | src type << 24 | dst type << 28
    __device__ int count() const { return (int)(info & 0xFFFFFFu); }
    __device__ int src_dtype() const { return (int)(info >> 24 & 15u); }
    __device__ int dst_dtype() const { return (int)(info >> 28); }
};
static_assert(sizeof(Piece) == 16, "one scalar load");

// Elements of a whole piece of the passes that write, and of a rest: with one
// 16-byte access per lane and row, a block has all of a piece in flight.
// 16384-element pieces ran at 5.3 TB/s where these run at 6.2 (accumulation of
// 9.4e8 bf16 into fp32: 1770 and 1506 us); with 4096 elements as four blocks to a
// larger record the tables of many small tensors were 15-20 % slower.
constexpr int kPiece = 4096;
// Elements of a run of the norm: 4096-element pieces, a wave each, read 6.7e9 bf16
// at 6.73 TB/s, runs by whole blocks at 6.97 (and 10,000 ragged tensors at 6.56
// with rests by waves, 6.37 by blocks; all four at 8 blocks per CU and groups of 1).
constexpr int kRun = 16384;
// Consecutive units an XCD gets of each.  Norm of 6.7e9 bf16: 1854 us at 16, 1878 at 8,
// 1837 at 32, 1935 to 1941 at 1 to 4; 10,000 ragged tensors 304 at 16, 303 at 8, 305 at
// 32, 311 at 1.  Clip of 9.4e8 bf16 in place: 566 us at 32, 561 at 16, 576 at 8, 583 at
// 1; accumulation into fp32 1449, 1443, 1449 and 1497.
constexpr int kRunGroup = 16, kPieceGroup = 32;
// Resident blocks per CU (lds_for_blocks).  Clip of 9.4e8 elements, at 3, 5 and 8: bf16 in
// place 686, 566 and 592 us, fp16 592, 562 and 575, fp32 into bf16 864, 885 and 903, fp32
// 1184, 1210 and 1242; 8.3e7 ragged bf16 72, 54 and 53.  The norm has 5, and 3 for
// large tables of aligned 16-bit tensors (norm_blocks); accumulation 2 to 8
// (add_blocks).
constexpr int kNormBlocksPerCU = 5, kClipBlocksPerCU = 5;
// Loads of 16 bytes that a lane has in flight in the norm of a run, and of a
// rest (8 for the runs: 1 % slower; 4 for the rests: the same).
constexpr int kRunLoads = 4, kRestLoads = 8;
constexpr int kWaves = kThreads / 64;

// Tensor pointers come out of the table; these types make the accesses global
// ones (not flat), at any element.
typedef __attribute__((address_space(1))) const char g_cbyte;
typedef __attribute__((address_space(1))) char g_byte;
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef __attribute__((address_space(1))) const u32x4_a2 g_cu32x4_a2;
typedef __attribute__((address_space(1))) u32x4_a2 g_u32x4_a2;
typedef __attribute__((address_space(1))) const u32x2_a2 g_cu32x2_a2;
typedef __attribute__((address_space(1))) u32x2_a2 g_u32x2_a2;
typedef __attribute__((address_space(1))) const uint32_t g_cu32;
typedef __attribute__((address_space(1))) const uint16_t g_cu16;
typedef __attribute__((address_space(1))) uint16_t g_u16;
typedef __attribute__((address_space(1))) const float g_cf32;
typedef __attribute__((address_space(1))) float g_f32;

template <int DT>
constexpr int kBytes = DT == ZERO_FP32 ? 4 : 2;

// --------------------------------------------------------- elements --------
template <int DT>
__device__ __forceinline__ float widen(uint16_t b) {
    return DT == ZERO_FP16 ? (float)__builtin_bit_cast(_Float16, b)
                           : __uint_as_float((uint32_t)b << 16);
}
// Nearest, ties to even; overflow gives inf, NaN stays (quiet) NaN.
template <int DT>
__device__ __forceinline__ uint16_t narrow(float f) {
    if (DT == ZERO_FP16) return __builtin_bit_cast(uint16_t, (_Float16)f);
    const uint32_t u = __float_as_uint(f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((u >> 16) | 0x0040u);
    return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}

// W (4 or 8) consecutive elements of a lane as they lie in memory.
template <int DT, int W>
struct Raw {
    static constexpr int kDwords = W * kBytes<DT> / 4;
    uint32_t w[kDwords];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int k = 0; k < kDwords; ++k) w[k] = 0;
    }
    __device__ __forceinline__ float get(int k) const {
        if constexpr (DT == ZERO_FP32) return __uint_as_float(w[k]);
        else return widen<DT>((uint16_t)((k & 1) ? (w[k >> 1] >> 16) : (w[k >> 1] & 0xFFFFu)));
    }
    __device__ __forceinline__ void set(int k, float v) {
        if constexpr (DT == ZERO_FP32) w[k] = __float_as_uint(v);
        else if (k & 1) w[k >> 1] |= (uint32_t)narrow<DT>(v) << 16;   // after the even one
        else w[k >> 1] = narrow<DT>(v);
    }
};
template <int DT, int W, bool NT>
__device__ __forceinline__ Raw<DT, W> load_raw(const void* p, int e) {
    Raw<DT, W> r;
    g_cbyte* b = (g_cbyte*)p + (int64_t)e * kBytes<DT>;
    if constexpr (Raw<DT, W>::kDwords == 2) {
        const u32x2 v = NT ? __builtin_nontemporal_load((g_cu32x2_a2*)b) : *(g_cu32x2_a2*)b;
        r.w[0] = v[0];
        r.w[1] = v[1];
    } else {
#pragma unroll
        for (int q = 0; q < Raw<DT, W>::kDwords / 4; ++q) {
            g_cu32x4_a2* c = (g_cu32x4_a2*)b + q;
            const u32x4 v = NT ? __builtin_nontemporal_load(c) : *c;
#pragma unroll
            for (int k = 0; k < 4; ++k) r.w[4 * q + k] = v[k];
        }
    }
    return r;
}
template <int DT, int W, bool NT>
__device__ __forceinline__ void store_raw(void* p, int e, const Raw<DT, W>& r) {
    g_byte* b = (g_byte*)p + (int64_t)e * kBytes<DT>;
    if constexpr (Raw<DT, W>::kDwords == 2) {
        const u32x2 v = {r.w[0], r.w[1]};
        if (NT) __builtin_nontemporal_store(v, (g_u32x2_a2*)b);
        else *(g_u32x2_a2*)b = v;
    } else {
#pragma unroll
        for (int q = 0; q < Raw<DT, W>::kDwords / 4; ++q) {
            g_u32x4_a2* c = (g_u32x4_a2*)b + q;
            const u32x4 v = {r.w[4 * q], r.w[4 * q + 1], r.w[4 * q + 2], r.w[4 * q + 3]};
            if (NT) __builtin_nontemporal_store(v, c);
            else *c = v;
        }
    }
}
template <int DT>
__device__ __forceinline__ float load_one(const void* p, int e) {
    if constexpr (DT == ZERO_FP32) return ((g_cf32*)p)[e];
    else return widen<DT>(((g_cu16*)p)[e]);
}
template <int DT>
__device__ __forceinline__ void store_one(void* p, int e, float v) {
    if constexpr (DT == ZERO_FP32) ((g_f32*)p)[e] = v;
    else ((g_u16*)p)[e] = narrow<DT>(v);
}

// The unit of work of block b of n: workgroups go to the 8 XCDs in turn, so blocks
// b, b + 8, ... of a group of 8 G share an XCD, and get G consecutive units.  The
// records of those then come from that XCD's L2 (handed out in order, every
// 128-byte line of records went to all 8: 3 % more bytes read by the clip) and
// the XCD reads memory in longer stretches.  Blocks past the last whole group
// keep their own.
template <int G>
__device__ __forceinline__ int64_t unit_of(int64_t b, int64_t n) {
    constexpr int64_t group = 8 * G;
    const int64_t a = b & ~(group - 1);
    if (a + group > n) return b;
    const int64_t r = b - a;
    return a + (r & 7) * G + (r >> 3);
}

template <int V>
struct Int {
    static constexpr int value = V;
};
// go(a type as an integral constant), for a piece's input, or output.
template <typename F>
__device__ __forceinline__ void by_type(int dtype, F&& go) {
    if (dtype == ZERO_FP32) go(Int<ZERO_FP32>{});
    else if (dtype == ZERO_FP16) go(Int<ZERO_FP16>{});
    else go(Int<ZERO_BF16>{});
}

// ------------------------------------------------------------ norms --------
// A running norm: the sum of squares, or the largest magnitude.  Magnitudes
// are compared as the bits of non-negative floats, which order as the values
// do with inf above them and NaN above inf, so a NaN anywhere is the result.
template <int KIND>
struct Norm {
    double s = 0.0;
    uint32_t m = 0;
    __device__ __forceinline__ void add(float x) {
        if (KIND == ZERO_NORM_L2) {
            const double d = (double)x;
            s = fma(d, d, s);                       // d * d is exact
        } else {
            const uint32_t b = __float_as_uint(x) & 0x7FFFFFFFu;
            m = b > m ? b : m;
        }
    }
    template <int DT, int W>
    __device__ __forceinline__ void add(const Raw<DT, W>& r) {
#pragma unroll
        for (int k = 0; k < W; ++k) add(r.get(k));
    }
    __device__ __forceinline__ double value() const {
        return KIND == ZERO_NORM_L2 ? s : (double)__uint_as_float(m);
    }
};

// Two partials joined: their sum, or the larger (NaN above all).
template <int KIND>
__device__ __forceinline__ double join(double a, double b) {
    if (KIND == ZERO_NORM_L2) return a + b;
    const uint64_t x = __builtin_bit_cast(uint64_t, a) & ~(uint64_t(1) << 63);
    const uint64_t y = __builtin_bit_cast(uint64_t, b) & ~(uint64_t(1) << 63);
    return __builtin_bit_cast(double, x > y ? x : y);
}
template <int KIND>
__device__ __forceinline__ double wave_join(double v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v = join<KIND>(v, __shfl_xor(v, off, 64));
    return v;
}
// The block's lanes joined, in a fixed order; valid in thread 0.
template <int KIND, int T = kThreads>
__device__ __forceinline__ double block_join(double v) {
    __shared__ double part[T / 64];
    v = wave_join<KIND>(v);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        v = part[0];
#pragma unroll
        for (int k = 1; k < T / 64; ++k) v = join<KIND>(v, part[k]);
    }
    return v;
}

// Thread t's share, of T, of the norm of a rest, U loads of 16 bytes in flight.
template <int KIND, int DT, int T, int U>
__device__ __forceinline__ double rest_norm(const void* src, int count, int t) {
    constexpr int W = 16 / kBytes<DT>, R = T * W;
    Norm<KIND> n;
    const int e = t * W;
    for (int b = 0; b < count; b += U * R) {
        Raw<DT, W> r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            r[u].clear();
            if (b + e + u * R + W <= count) r[u] = load_raw<DT, W, true>(src, b + e + u * R);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) n.add(r[u]);
    }
    const int last = count / W * W + t;
    if (last < count) n.add(load_one<DT>(src, last));
    return n.value();
}

// The thread's share of the norm of a run (exactly kRun elements), a block's work: a
// wave takes kRunLoads rows of 64 accesses, one after the other in memory, in each
// batch.  ODD: a 16-bit run that begins in the middle of a dword.  Accesses that
// are not aligned to a dword run at three quarters of the rate (1.07e9 fp16: 390 us,
// 300 at every other start and this way), so the dwords that hold the elements are
// read and shifted by one element, which puts every element where it would be
// otherwise.  A lane's last dword is the next lane's first, the last lane's is the
// next row's first, and only the batch's last is read for itself.  The dwords at
// the ends hold an element of the run each, so no access leaves the tensor's
// dwords.
template <int KIND, int DT, bool ODD>
__device__ __forceinline__ double run_norm(const void* src) {
    constexpr int W = 16 / kBytes<DT>, S = 64 * W, U = kRunLoads, B = kWaves * U * S;
    static_assert(kRun % B == 0, "whole batches");
    const int lane = threadIdx.x & 63;
    g_cbyte* p = (g_cbyte*)src - (ODD ? 2 : 0);
    const int e = (threadIdx.x >> 6) * U * S + lane * W;
    Norm<KIND> n;
#pragma unroll
    for (int b = 0; b < kRun; b += B) {
        Raw<DT, W> r[U];
        uint32_t tail = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) r[u] = load_raw<DT, W, true>((const void*)p, b + e + u * S);
        if constexpr (ODD) {
            if (lane == 63) tail = *(g_cu32*)(p + (b + e + (U - 1) * S + W) * 2);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // the next lane's first dword (a DPP wave shift), or the next row's
                const uint32_t next = (uint32_t)__builtin_amdgcn_update_dpp(
                    0, (int)r[u].w[0], 0x130 /* wave_shl:1 */, 0xF, 0xF, false);
                const uint32_t row = u + 1 < U
                    ? (uint32_t)__builtin_amdgcn_readfirstlane((int)r[u + 1 < U ? u + 1 : u].w[0])
                    : tail;
                const uint32_t last = lane == 63 ? row : next;
#pragma unroll
                for (int k = 0; k < W / 2; ++k)
                    r[u].w[k] = __builtin_amdgcn_alignbit(k + 1 < W / 2 ? r[u].w[k + 1] : last,
                                                          r[u].w[k], 16);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) n.add(r[u]);
    }
    return n.value();
}

// One partial per run, a block each, then one per rest, a wave each.
template <int KIND>
__global__ void __launch_bounds__(kThreads)
tensor_norm_kernel(const Piece* __restrict__ runs, int64_t n_runs, int64_t n_rests, int64_t blk0,
                   double* __restrict__ part) {
    const int64_t b = blk0 + blockIdx.x;
    double v = 0.0;
    if (b < n_runs) {
        const int64_t i = unit_of<kRunGroup>(b, n_runs);
        const Piece p = runs[i];
        by_type(p.src_dtype(), [&](auto s) {
            constexpr int DT = decltype(s)::value;
            if constexpr (DT != ZERO_FP32)
                if ((uintptr_t)p.src & 2) {
                    v = run_norm<KIND, DT, true>(p.src);
                    return;
                }
            v = run_norm<KIND, DT, false>(p.src);
        });
        v = block_join<KIND>(v);
        if (threadIdx.x == 0) part[i] = v;
        return;
    }
    const int64_t i = (b - n_runs) * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (i >= n_rests) return;
    const Piece p = runs[n_runs + i];
    const int lane = threadIdx.x & 63;
    by_type(p.src_dtype(), [&](auto s) {
        v = rest_norm<KIND, decltype(s)::value, 64, kRestLoads>(p.src, p.count(), lane);
    });
    v = wave_join<KIND>(v);
    if (lane == 0) part[n_runs + i] = v;
}

// Thread `t` of T's share of part[0, n): part[t], part[t + T], ..., kInFlight
// loads at a time.
constexpr int kInFlight = 16;
template <int KIND, int T>
__device__ __forceinline__ double strided_join(const double* __restrict__ part, int64_t n, int t) {
    double v = 0.0;
    for (int64_t b = 0; b < n; b += kInFlight * T) {
        double x[kInFlight];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            const int64_t j = b + u * T + t;
            x[u] = j < n ? part[j] : 0.0;
        }
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) v = join<KIND>(v, x[u]);
    }
    return v;
}

// Block b joins partials [b * kFoldEach, (b + 1) * kFoldEach).
constexpr int kFoldEach = kInFlight * kThreads;
template <int KIND>
__global__ void __launch_bounds__(kThreads)
tensor_fold_kernel(const double* __restrict__ part, int64_t n, double* __restrict__ out) {
    const int64_t a = (int64_t)blockIdx.x * kFoldEach;
    const int64_t left = n - a < kFoldEach ? n - a : kFoldEach;
    const double v = block_join<KIND>(strided_join<KIND, kThreads>(part + a, left, threadIdx.x));
    if (threadIdx.x == 0) out[blockIdx.x] = v;
}

// The result for a joined norm v, and its way into *res.
template <int KIND>
__device__ __forceinline__ zero_step_result result_of(double v, float inv) {
    zero_step_result r;
    const double x = KIND == ZERO_NORM_L2 ? v : v * v;
    r.sumsq = x * ((double)inv * (double)inv);
    r.overflow = x < INFINITY ? 0u : 1u;              // NaN and inf are not
    r.inv_scale = inv;
    return r;
}
template <int KIND>
__device__ __forceinline__ void store_result(zero_step_result r, int accumulate,
                                             zero_step_result* res) {
    if (accumulate) {
        r.overflow |= res->overflow;
        r.sumsq = join<KIND>(res->sumsq, r.sumsq);
    }
    *res = r;
}

template <int KIND>
__device__ __forceinline__ float tensor_norm(double v, float inv) {
    return (float)((KIND == ZERO_NORM_L2 ? sqrt(v) : v) * (double)inv);
}

// Block 0 joins the n (folded) partials into *res; the others join each tensor's
// partials, which are at first[t] to first[t + 1] and (where given) first2[t]
// to first2[t + 1], into norms, T threads to a tensor.
constexpr int kFinishThreads = 1024;
template <int KIND, int T>
__global__ void __launch_bounds__(kFinishThreads)
tensor_finish_kernel(const double* __restrict__ part, int64_t n,
                     const double* __restrict__ tensor_part, const int64_t* __restrict__ first,
                     const int64_t* __restrict__ first2, int64_t n_tensors, float inv_scale,
                     const zero_step_control* __restrict__ ctl, int accumulate,
                     zero_step_result* res, float* __restrict__ norms) {
    const float inv = ctl ? ctl->inv_scale : inv_scale;
    if (blockIdx.x == 0) {
        const double v = block_join<KIND, kFinishThreads>(
            strided_join<KIND, kFinishThreads>(part, n, threadIdx.x));
        if (threadIdx.x == 0) store_result<KIND>(result_of<KIND>(v, inv), accumulate, res);
        return;
    }
    const int64_t t = ((int64_t)blockIdx.x - 1) * (kFinishThreads / T) +
                      __builtin_amdgcn_readfirstlane(threadIdx.x / T);
    if (t >= n_tensors) return;                       // whole waves, or the whole block
    const int64_t a = first[t];
    double v = strided_join<KIND, T>(tensor_part + a, first[t + 1] - a, threadIdx.x % T);
    if (first2) {
        const int64_t a2 = first2[t];
        v = join<KIND>(v, strided_join<KIND, T>(tensor_part + a2, first2[t + 1] - a2, threadIdx.x % T));
    }
    if (T == kFinishThreads) v = block_join<KIND, kFinishThreads>(v);
    else v = wave_join<KIND>(v);
    if (threadIdx.x % T == 0) norms[t] = tensor_norm<KIND>(v, inv);
}

// ------------------------------------------------------------- clip --------
// max_norm / (norm + 1e-6) where that is below 1, else 1 (a NaN norm: 1), times
// the unscale factor; fp64, rounded once; never NaN.
__device__ __forceinline__ float clip_factor(float max_norm, double norm, float inv) {
    double c = 1.0;
    if (max_norm > 0.0f) {
        const double q = (double)max_norm / (norm + 1e-6);
        if (q < 1.0) c = q;
    }
    return (float)(c * (double)inv);
}

// Elements per lane access of a pass that reads SRC and writes DST: 16 bytes of
// the wider of the two, so that a wave's access is one stretch (with 8 elements,
// two accesses 16 bytes apart on the fp32 side, accumulations into fp32 took 1822
// us for 1765 and, over ragged tables, 216 for 196).
template <int SRC, int DST>
constexpr int kWidth = kBytes<SRC> == 4 || kBytes<DST> == 4 ? 4 : 8;

// factor() is called after the loads are issued: its fp64 root and division
// overlap their latency.  It is NaN where the step is skipped.  NT: loads that do
// not stay in the caches.
template <int SRC, int DST, bool NT, int T, typename F>
__device__ __forceinline__ void piece_scale(const void* src, void* dst, int count, F&& factor) {
    constexpr int W = kWidth<SRC, DST>, R = W * T, U = (kPiece + R - 1) / R;
    const int e = threadIdx.x * W;
    auto scaled = [](const Raw<SRC, W>& x, float f) {
        Raw<DST, W> y;
#pragma unroll
        for (int k = 0; k < W; ++k) y.set(k, x.get(k) * f);
        return y;
    };
    // a skipped step, or in place with a factor of 1 (900 tensors of 16384 fp32: norm
    // and clip 22.9 us for 31.5): nothing to write, though it has been read
    auto nothing = [&](float f) { return f != f || (SRC == DST && f == 1.0f && src == dst); };
    Raw<SRC, W> r[U];
    if (U * R == kPiece && count == kPiece) {
#pragma unroll
        for (int u = 0; u < U; ++u) r[u] = load_raw<SRC, W, NT>(src, e + u * R);
        const float f = factor();
        if (nothing(f)) return;
#pragma unroll
        for (int u = 0; u < U; ++u) store_raw<DST, W, true>(dst, e + u * R, scaled(r[u], f));
        return;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (e + u * R + W <= count) r[u] = load_raw<SRC, W, NT>(src, e + u * R);
    const int t = count / W * W + threadIdx.x;
    const float last = t < count ? load_one<SRC>(src, t) : 0.0f;
    const float f = factor();
    if (nothing(f)) return;
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (e + u * R + W <= count) store_raw<DST, W, true>(dst, e + u * R, scaled(r[u], f));
    if (t < count) store_one<DST>(dst, t, last * f);
}
template <bool NT, int T, typename F>
__device__ __forceinline__ void scale_by_types(const Piece& p, void* dst, F&& factor) {
    by_type(p.src_dtype(), [&](auto s) {
        by_type(p.dst_dtype(), [&](auto d) {
            piece_scale<decltype(s)::value, decltype(d)::value, NT, T>(p.src, dst, p.count(), factor);
        });
    });
}

template <bool NT>
__global__ void __launch_bounds__(kThreads)
tensor_clip_kernel(const Piece* __restrict__ pieces, void* const* __restrict__ dsts, float max_norm,
                   const zero_step_result* __restrict__ res, const float* __restrict__ norms) {
    const int64_t i = unit_of<kPieceGroup>(blockIdx.x, gridDim.x);
    const Piece p = pieces[i];
    void* dst = dsts[i];
    const zero_step_result r = *res;
    if (r.overflow) return;                          // skipped step: write nothing
    // In place with a factor of 1 there is nothing to write either (9.4e8 bf16: 68
    // us instead of 566).  The test costs no root: a norm of at most max_norm - 1e-6
    // gives a ratio that is 1 or more, or rounds to 1.
    if (p.src == dst && p.src_dtype() == p.dst_dtype() && r.inv_scale == 1.0f) {
        const double most = (double)max_norm - 1e-6;
        if (max_norm <= 0.0f || (most > 0.0 && (norms ? (double)norms[p.tensor] <= most
                                                      : r.sumsq <= most * most)))
            return;
    }
    scale_by_types<NT, kThreads>(p, dst, [&] {
        return clip_factor(max_norm, norms ? (double)norms[p.tensor] : sqrt(r.sumsq), r.inv_scale);
    });
}

// The clip right after the partials of a norm, at most kJoinPartials: every block
// joins them itself (in the order of tensor_finish_kernel, so to the same
// bits), which spares that launch; the block of piece 0 stores the result.
// 60 tensors of 16384 fp32: 8.9 us against 12.0 with the launch; at 1000 of them
// (1000 partials) 35.0 against 36.6.
constexpr int kJoinPartials = 1024;
static_assert(kJoinPartials == kFinishThreads && kJoinPartials % kThreads == 0,
              "the finishing block's one partial per thread");
template <int KIND>
__global__ void __launch_bounds__(kThreads)
tensor_join_clip_kernel(const Piece* __restrict__ pieces, void* const* __restrict__ dsts,
                        float max_norm, const double* __restrict__ part, int n, float inv_scale,
                        const zero_step_control* __restrict__ ctl, zero_step_result* res) {
    __shared__ double joined[kJoinPartials / 64];
    const int64_t i = unit_of<kPieceGroup>(blockIdx.x, gridDim.x);
    const Piece p = pieces[i];
    scale_by_types<false, kThreads>(p, dsts[i], [&] {
        double x[kJoinPartials / kThreads];
#pragma unroll
        for (int q = 0; q < kJoinPartials / kThreads; ++q) {
            const int j = q * kThreads + threadIdx.x;
            x[q] = j < n ? part[j] : 0.0;
        }
        const float inv = ctl ? ctl->inv_scale : inv_scale;
#pragma unroll
        for (int q = 0; q < kJoinPartials / kThreads; ++q) {
            x[q] = wave_join<KIND>(x[q]);
            if ((threadIdx.x & 63) == 0) joined[q * kWaves + (threadIdx.x >> 6)] = x[q];
        }
        __syncthreads();
        double v = joined[0];
#pragma unroll
        for (int k = 1; k < kJoinPartials / 64; ++k) v = join<KIND>(v, joined[k]);
        const zero_step_result r = result_of<KIND>(v, inv);
        if (i == 0 && threadIdx.x == 0) *res = r;
        return r.overflow ? NAN : clip_factor(max_norm, sqrt(r.sumsq), inv);
    });
}

// Norm, each tensor's norm and (CLIP) the clip of a table of at most kOneBlock
// rests and no run (and, with norms, few tensors), in one block, which joins in the order of
// tensor_finish_kernel (a wave's tree over at most 64 partials), so to the same
// bits.
constexpr int kOneBlock = kFinishThreads / 64;       // a wave for each rest
template <int KIND, bool CLIP>
__global__ void __launch_bounds__(kFinishThreads)
tensor_one_block_kernel(const Piece* __restrict__ rests, int n_rests,
                        const Piece* __restrict__ pieces, void* const* __restrict__ dsts, int n_pieces,
                        const int64_t* __restrict__ first, int64_t n_tensors, float max_norm,
                        int per_tensor, float inv_scale, const zero_step_control* __restrict__ ctl,
                        int accumulate, zero_step_result* res, float* __restrict__ norms) {
    __shared__ double part[64];
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    double v = 0.0;
    if (w < n_rests) {
        const Piece p = rests[w];
        by_type(p.src_dtype(), [&](auto s) {
            v = rest_norm<KIND, decltype(s)::value, 64, kRestLoads>(p.src, p.count(), lane);
        });
    }
    v = wave_join<KIND>(v);
    if (lane == 0) part[w] = v;
    const float inv = ctl ? ctl->inv_scale : inv_scale;
    __syncthreads();
    auto joined = [&](int a, int n) {                 // by a whole wave
        return wave_join<KIND>(lane < n ? part[a + lane] : 0.0);
    };
    auto norm_of = [&](int64_t t) {
        return tensor_norm<KIND>(joined((int)first[t], (int)(first[t + 1] - first[t])), inv);
    };
    const zero_step_result r = result_of<KIND>(joined(0, n_rests), inv);
    if (threadIdx.x == 0) store_result<KIND>(r, accumulate, res);
    if (norms)
        for (int64_t t = w; t < n_tensors; t += kFinishThreads / 64) {
            const float x = norm_of(t);
            if (lane == 0) norms[t] = x;
        }
    if (!CLIP || r.overflow) return;
    for (int k = 0; k < n_pieces; ++k) {
        const Piece p = pieces[k];
        const double norm = per_tensor ? (double)norm_of(p.tensor) : sqrt(r.sumsq);
        scale_by_types<false, kFinishThreads>(p, dsts[k],
                                              [&] { return clip_factor(max_norm, norm, inv); });
    }
}

// ------------------------------------------------------- accumulate --------
// KIND 0: no norm of the result.  Loads and stores that do not stay in the caches:
// 1736 us with plain ones for 9.4e8 bf16 into fp32, against 1501; a table of 83 MB
// gains 6 % from plain ones, of 221 MB loses 13 %.
template <int KIND, bool FIRST, int SRC, int DST>
__device__ __forceinline__ void piece_accumulate(const void* src, void* dst, int count, float w,
                                                 Norm<KIND>& n) {
    constexpr int W = kWidth<SRC, DST>, R = W * kThreads, U = kPiece / R;
    const int e = threadIdx.x * W;
    Raw<SRC, W> x[U];
    Raw<DST, W> y[U];
    auto load = [&](int u) {
        x[u] = load_raw<SRC, W, true>(src, e + u * R);
        if (FIRST) y[u].clear();
        else y[u] = load_raw<DST, W, true>(dst, e + u * R);
    };
    auto add = [&](int u) {
        Raw<DST, W> z;
#pragma unroll
        for (int k = 0; k < W; ++k) {
            z.set(k, FIRST ? w * x[u].get(k) : fmaf(w, x[u].get(k), y[u].get(k)));
            if (KIND) n.add(z.get(k));               // what a pass over dst would read
        }
        store_raw<DST, W, true>(dst, e + u * R, z);
    };
    if (count == kPiece) {
#pragma unroll
        for (int u = 0; u < U; ++u) load(u);
#pragma unroll
        for (int u = 0; u < U; ++u) add(u);
        return;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (e + u * R + W <= count) load(u);
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (e + u * R + W <= count) add(u);
    const int t = count / W * W + threadIdx.x;
    if (t < count) {
        const float a = load_one<SRC>(src, t);
        const float v = FIRST ? w * a : fmaf(w, a, load_one<DST>(dst, t));
        store_one<DST>(dst, t, v);
        if (KIND) {
            Raw<DST, 4> z;                           // v as stored
            z.set(0, v);
            n.add(z.get(0));
        }
    }
}

template <int KIND, bool FIRST>
__global__ void __launch_bounds__(kThreads)
tensor_accumulate_kernel(const Piece* __restrict__ pieces, void* const* __restrict__ dsts, float w,
                         double* __restrict__ part) {
    const int64_t i = unit_of<kPieceGroup>(blockIdx.x, gridDim.x);
    const Piece p = pieces[i];
    void* dst = dsts[i];
    Norm<KIND> n;
    by_type(p.src_dtype(), [&](auto s) {
        by_type(p.dst_dtype(), [&](auto d) {
            piece_accumulate<KIND, FIRST, decltype(s)::value, decltype(d)::value>(p.src, dst, p.count(),
                                                                                 w, n);
        });
    });
    if (KIND) {
        const double v = block_join<KIND>(n.value());
        if (threadIdx.x == 0) part[i] = v;
    }
}

// ------------------------------------------------------------ table --------
__host__ __device__ inline int64_t dtype_bytes(int32_t dt) { return dt == ZERO_FP32 ? 4 : 2; }

// Elements of a tensor's first piece: the others then begin at a multiple of
// 128 bytes of the output.
__host__ __device__ inline int64_t first_piece(const zero_tensor_entry& e) {
    return kPiece - (int64_t)((uintptr_t)e.dst % 128) / dtype_bytes(e.dst_dtype);
}
__host__ __device__ inline int64_t runs_in(const zero_tensor_entry& e) { return e.numel / kRun; }
__host__ __device__ inline int64_t rests_in(const zero_tensor_entry& e) {
    return (e.numel % kRun + kPiece - 1) / kPiece;
}
__host__ __device__ inline int64_t pieces_in(const zero_tensor_entry& e) {
    if (e.numel == 0) return 0;
    const int64_t first = first_piece(e);
    return e.numel <= first ? 1 : 1 + (e.numel - first - 1) / kPiece + 1;
}

// Last index k of first[0, n] (ascending, first[0] <= u < first[n]) with
// first[k] <= u: the tensor that holds unit u.
__device__ __forceinline__ int64_t holder(const int64_t* __restrict__ first, int64_t n, int64_t u) {
    int64_t lo = 0, hi = n;                           // first[lo] <= u < first[hi]
    while (hi - lo > 1) {
        const int64_t mid = lo + (hi - lo) / 2;
        if (first[mid] <= u) lo = mid;
        else hi = mid;
    }
    return lo;
}

// A thread for each record of the table.
__global__ void __launch_bounds__(kThreads)
tensor_expand_kernel(const zero_tensor_entry* __restrict__ entries,
                     const int64_t* __restrict__ first_run, const int64_t* __restrict__ first_rest,
                     const int64_t* __restrict__ first_piece_at, int64_t n, int64_t n_runs,
                     int64_t n_rests, int64_t n_pieces, int64_t blk0, Piece* __restrict__ runs,
                     Piece* __restrict__ pieces, void** __restrict__ dsts) {
    const int64_t u = (blk0 + blockIdx.x) * kThreads + threadIdx.x;
    const int64_t q = u - n_runs - n_rests;           // piece
    if (q >= n_pieces) return;
    const int64_t* first = u < n_runs ? first_run : q < 0 ? first_rest : first_piece_at;
    const int64_t k = holder(first, n, q < 0 ? u : q);
    const zero_tensor_entry e = entries[k];
    const int64_t j = (q < 0 ? u : q) - first[k];     // of the tensor's
    int64_t begin, most;
    if (u < n_runs) {
        begin = j * kRun;
        most = kRun;
    } else if (q < 0) {
        begin = runs_in(e) * kRun + j * kPiece;
        most = kPiece;
    } else {
        const int64_t f = first_piece(e);
        begin = j == 0 ? 0 : f + (j - 1) * kPiece;
        most = j == 0 ? f : kPiece;
    }
    const int64_t left = e.numel - begin;
    Piece p;
    p.src = (const char*)e.src + begin * dtype_bytes(e.src_dtype);
    p.tensor = (int32_t)k;
    p.info = (uint32_t)(left < most ? left : most) | (uint32_t)e.src_dtype << 24 |
             (uint32_t)e.dst_dtype << 28;
    if (q < 0) {
        runs[u] = p;
    } else {
        pieces[q] = p;
        dsts[q] = (char*)e.dst + begin * dtype_bytes(e.dst_dtype);
    }
}

// ------------------------------------------------------------- host --------
inline bool valid_table_dtype(int32_t dt) { return valid_dtype(dt) || dt == ZERO_FP32; }

// Tensors of a plan: one launch finishes a norm for each.
constexpr int64_t kMaxTensors = kMaxLaunchBlocks;

struct Span {
    uintptr_t begin, end;
};

// One side of an entry as a span of addresses; false where it is not one.
bool span_of(const void* p, int64_t numel, int32_t dtype, Span* s) {
    uintptr_t bytes;
    s->begin = s->end = (uintptr_t)p;
    if (__builtin_mul_overflow((uintptr_t)numel, (uintptr_t)dtype_bytes(dtype), &bytes)) return false;
    return !__builtin_add_overflow(s->begin, bytes, &s->end);
}

bool overlaps(const std::vector<Span>& sorted, const Span& s) {
    // `sorted`: disjoint spans in order; most inputs lie beyond all outputs, others are
    // compared with the first that ends after s begins
    if (sorted.empty() || s.end <= sorted.front().begin || sorted.back().end <= s.begin) return false;
    auto it = std::upper_bound(sorted.begin(), sorted.end(), s.begin,
                               [](uintptr_t a, const Span& b) { return a < b.end; });
    return it != sorted.end() && it->begin < s.end;
}

// Whether a call may write the table's outputs: no output overlaps another,
// nor an input other than its own at the same address and of the same type.
bool writable(const zero_tensor_entry* entries, int64_t n) {
    std::vector<Span> out;
    out.reserve((size_t)n);
    Span s;
    for (int64_t k = 0; k < n; ++k)
        if (entries[k].numel > 0 && span_of(entries[k].dst, entries[k].numel, entries[k].dst_dtype, &s))
            out.push_back(s);
    const auto before = [](const Span& a, const Span& b) { return a.begin < b.begin; };
    if (!std::is_sorted(out.begin(), out.end(), before)) std::sort(out.begin(), out.end(), before);
    for (size_t k = 1; k < out.size(); ++k)
        if (out[k].begin < out[k - 1].end) return false;
    for (int64_t k = 0; k < n; ++k) {
        const zero_tensor_entry& e = entries[k];
        if (e.numel <= 0 || (e.src == e.dst && e.src_dtype == e.dst_dtype)) continue;
        if (span_of(e.src, e.numel, e.src_dtype, &s) && overlaps(out, s)) return false;
    }
    return true;
}

// More pieces than any memory holds whole tensors of, and few enough for every
// size computed from them.
constexpr int64_t kMaxPieces = int64_t(1) << 40;

int plan_of(const zero_tensor_entry* entries, int64_t n, zero_tensor_plan* plan) {
    int64_t numel = 0, bytes = 0, fp32_out = 0, even16 = 0, pieces = 0, runs = 0, rests = 0, largest = 0;
    for (int64_t k = 0; k < n; ++k) {
        const zero_tensor_entry& e = entries[k];
        if (e.numel < 0 || !valid_table_dtype(e.src_dtype) || !valid_table_dtype(e.dst_dtype))
            return ZERO_EINVAL;
        if (e.numel == 0) continue;
        if (!e.src || !e.dst) return ZERO_EINVAL;
        if ((uintptr_t)e.src % (uintptr_t)dtype_bytes(e.src_dtype) ||
            (uintptr_t)e.dst % (uintptr_t)dtype_bytes(e.dst_dtype))
            return ZERO_EINVAL;
        Span s;
        if (!span_of(e.src, e.numel, e.src_dtype, &s) || !span_of(e.dst, e.numel, e.dst_dtype, &s))
            return ZERO_ERANGE;
        if (pieces_in(e) > kMaxPieces - pieces) return ZERO_ERANGE;
        pieces += pieces_in(e);
        if (__builtin_add_overflow(numel, e.numel, &numel) ||
            __builtin_add_overflow(bytes, e.numel * (dtype_bytes(e.src_dtype) + dtype_bytes(e.dst_dtype)),
                                   &bytes))
            return ZERO_ERANGE;
        if (e.dst_dtype == ZERO_FP32) fp32_out += e.numel;
        if (e.src_dtype != ZERO_FP32 && (uintptr_t)e.src % 4 == 0) even16 += e.numel;
        runs += runs_in(e);
        rests += rests_in(e);
        largest = std::max(largest, e.numel / kPiece);
    }
    plan->n_tensors = n;
    plan->numel = numel;
    plan->bytes = bytes;
    plan->n_pieces = pieces;
    plan->n_runs = runs;
    plan->n_rests = rests;
    plan->head_bytes = (n * (int64_t)sizeof(zero_tensor_entry) + 3 * (n + 1) * (int64_t)sizeof(int64_t) +
                        15) / 16 * 16;
    plan->table_bytes = plan->head_bytes + (pieces + runs + rests) * (int64_t)sizeof(Piece) +
                        pieces * (int64_t)sizeof(void*);
    plan->fp32_out = fp32_out > numel / 2 ? 1 : 0;
    plan->even16 = numel > 0 && even16 >= numel / 8 * 7 ? 1 : 0;
    plan->largest = (int32_t)std::min<int64_t>(largest, INT32_MAX);
    try {
        plan->writable = writable(entries, n) ? 1 : 0;
    } catch (const std::bad_alloc&) {
        return ZERO_ERANGE;
    }
    return ZERO_OK;
}

// What a device call needs of a plan and its table.
bool valid_plan(const zero_tensor_plan* p, const void* table) {
    return p && p->n_tensors >= 0 && p->n_tensors < kMaxTensors && p->n_pieces >= 0 &&
           p->n_pieces <= kMaxPieces && p->n_runs >= 0 && p->n_rests >= 0 && p->n_runs <= p->n_pieces &&
           p->n_rests <= p->n_pieces && p->head_bytes >= 0 && table && ((uintptr_t)table & 15) == 0;
}

// The parts of a table, in its order.  The head: the entries, and for every tensor
// (and the end) its first run's partial, first rest's partial and first piece.
// Then the norm's runs and rests, the pieces of the passes that write and their
// outputs.
const zero_tensor_entry* entries_of(const void* table) { return (const zero_tensor_entry*)table; }
const int64_t* first_runs_of(const zero_tensor_plan* p, const void* table) {
    return (const int64_t*)(entries_of(table) + p->n_tensors);
}
const int64_t* first_rests_of(const zero_tensor_plan* p, const void* table) {
    return first_runs_of(p, table) + p->n_tensors + 1;
}
const int64_t* first_pieces_of(const zero_tensor_plan* p, const void* table) {
    return first_rests_of(p, table) + p->n_tensors + 1;
}
const Piece* runs_of(const zero_tensor_plan* p, const void* table) {
    return (const Piece*)((const char*)table + p->head_bytes);
}
const Piece* pieces_of(const zero_tensor_plan* p, const void* table) {
    return runs_of(p, table) + p->n_runs + p->n_rests;
}
void* const* dsts_of(const zero_tensor_plan* p, const void* table) {
    return (void* const*)(pieces_of(p, table) + p->n_pieces);
}

// Partials that the finishing block takes as they are; more are folded first (20,000
// of them: a norm of 17.0 us, 17.6 with a fold; 40,000: 30.1 without, 28.8 with).
constexpr int64_t kFinish = 2 * kInFlight * kFinishThreads;
int64_t fold_blocks(int64_t n) { return n <= kFinish ? 0 : (n + kFoldEach - 1) / kFoldEach; }

// Runs `blocks` blocks as launches of at most kMaxLaunchBlocks, in order:
// go(first block, blocks).
template <typename F>
int in_launches(int64_t blocks, F&& go) {
    for (int64_t b = 0; b < blocks; b += kMaxLaunchBlocks) {
        const int rc = go(b, std::min(kMaxLaunchBlocks, blocks - b));
        if (rc != ZERO_OK) return rc;
    }
    return ZERO_OK;
}

int norm_args(const zero_tensor_plan* plan, const void* table, int32_t kind, float inv_scale,
              const zero_step_control* ctl, const zero_step_result* res, const void* workspace,
              size_t workspace_bytes) {
    if (!valid_plan(plan, table) || (kind != ZERO_NORM_L2 && kind != ZERO_NORM_MAX)) return ZERO_EINVAL;
    if (!res || !workspace || ((uintptr_t)workspace & 7) != 0) return ZERO_EINVAL;
    if (!ctl && (!(inv_scale > 0.0f) || !__builtin_isfinite(inv_scale))) return ZERO_EINVAL;
    if (workspace_bytes < zero_tensor_workspace_bytes(plan)) return ZERO_EINVAL;
    return ZERO_OK;
}

// Joins the n partials at the workspace's start into *res and norms; `most`: those of
// the largest tensor.
template <int KIND>
int finish(int64_t n, int64_t most, const int64_t* first, const int64_t* first2, int64_t n_tensors,
           float inv_scale, const zero_step_control* ctl, int32_t accumulate, zero_step_result* res,
           float* norms, double* part, hipStream_t stream) {
    const double* last = part;
    const int64_t nt = norms ? n_tensors : 0;
    // A block for each tensor, or a wave.  A wave takes 1024 of a tensor's partials a round
    // (0.5 us each), so the largest tensor decides; blocks take 3.6 us more per 1000
    // tensors.  Norm with each tensor's, block and wave: 1.1e9 bf16 beside 100 tensors
    // of 64: 299 and 334 us, beside 5000: 318 and 337, beside 20,000: 388 and 346; 2.7e8
    // beside 1000: 81 and 87; 6.7e7 beside 1000: 26.9 and 25.2.  (The last condition: a
    // launch's threads are counted in 32 bits.)
    const bool wide = most > 1024 && most > 8 * nt &&
                      nt < kMaxLaunchBlocks / (kFinishThreads / kThreads);
    if (const int64_t blocks = fold_blocks(n)) {
        const int rc = launch(tensor_fold_kernel<KIND>, blocks, 0, stream, part, n, part + n);
        if (rc != ZERO_OK) return rc;
        last = part + n;
        n = blocks;
    }
    const auto kernel = wide ? tensor_finish_kernel<KIND, kFinishThreads>
                             : tensor_finish_kernel<KIND, 64>;
    const int64_t each = wide ? 1 : kFinishThreads / 64;
    return launch_shape(kernel, 1 + (nt + each - 1) / each, kFinishThreads, 0u, stream, last, n, part,
                        first, first2, nt, inv_scale, ctl, (int)(accumulate != 0), res, norms);
}

// Whether a table's norm takes one block (16 tensors of 4096 fp32: 6.1 us against
// 8.8 for two launches), and its norm and clip together, which that block does
// one piece after the other (4: 6.6 us against 8.7, 8: 8.8, 16: 13.3 against 8.6).
// Its 16 waves take the tensors' own norms in turn, so these are few too (empty tensors
// count here alone).  Norm and every tensor's of 128 of which one holds elements: 7.6
// us against 9.0, 256: 12.1 against 8.7, 200,000: 8250 against 45; with the clip 8.5
// against 12.5, and 13.1 against 12.4 at 256.
constexpr int kOneBlockPieces = 4;
constexpr int64_t kOneBlockTensors = 128;
bool one_block(const zero_tensor_plan* p, const float* norms) {
    return p->n_runs == 0 && p->n_rests <= kOneBlock && (!norms || p->n_tensors <= kOneBlockTensors);
}
bool one_block_clip(const zero_tensor_plan* p, const float* norms) {
    return one_block(p, norms) && p->n_pieces <= kOneBlockPieces;
}

template <int KIND, bool CLIP>
int one_block_impl(const zero_tensor_plan* plan, const void* table, float max_norm,
                   int32_t per_tensor, float inv_scale, const zero_step_control* ctl,
                   int32_t accumulate, zero_step_result* res, float* norms, hipStream_t stream) {
    return launch_shape(tensor_one_block_kernel<KIND, CLIP>, 1, kFinishThreads, 0u, stream,
                        runs_of(plan, table), (int)plan->n_rests, pieces_of(plan, table),
                        dsts_of(plan, table), (int)plan->n_pieces, first_rests_of(plan, table),
                        plan->n_tensors, max_norm, (int)(per_tensor != 0), inv_scale, ctl,
                        (int)(accumulate != 0), res, norms);
}

// Resident blocks per CU of the norm.  16-bit tensors that begin at a dword: 6.7e9
// elements take 1851 us at 3, 1908 at 5 and at 8; 9.4e8 256 and 272; 4.4e8 127 and 131;
// 2.2e8 65 and 68; 1.4e8 the same.  10,000 packed tensors, half of which begin between
// dwords: 325 at 3, 304 at 5; ragged ones of 8.3e7 33 and 31; fp32 the same to 1 %.
int norm_blocks(const zero_tensor_plan* p) {
    return p->even16 && p->n_runs >= 16384 ? 3 : kNormBlocksPerCU;
}

// The partials of the norm, runs first.
template <int KIND>
int partials_impl(const zero_tensor_plan* plan, const void* table, double* part, hipStream_t stream) {
    const int64_t n_runs = plan->n_runs, n_rests = plan->n_rests;
    return in_launches(n_runs + (n_rests + kWaves - 1) / kWaves, [&](int64_t b, int64_t grid) {
        return launch(tensor_norm_kernel<KIND>, grid, lds_for_blocks(norm_blocks(plan)), stream,
                      runs_of(plan, table), n_runs, n_rests, b, part);
    });
}

template <int KIND>
int norm_impl(const zero_tensor_plan* plan, const void* table, float inv_scale,
              const zero_step_control* ctl, int32_t accumulate, zero_step_result* res, float* norms,
              double* part, hipStream_t stream) {
    if (one_block(plan, norms))
        return one_block_impl<KIND, false>(plan, table, 0.0f, 0, inv_scale, ctl, accumulate, res, norms,
                                           stream);
    const int rc = partials_impl<KIND>(plan, table, part, stream);
    if (rc != ZERO_OK) return rc;
    return finish<KIND>(plan->n_runs + plan->n_rests, plan->largest / (kRun / kPiece),
                        first_runs_of(plan, table), first_rests_of(plan, table), plan->n_tensors,
                        inv_scale, ctl, accumulate, res, norms, part, stream);
}

// Whether a clip reads and writes more than the last-level cache holds (256 MB): it
// then loads its inputs so that they do not stay there.  Three tables in turn: 202 MB
// read and written 36.1 us so, 31.5 us with plain loads; 401 MB 63.5 and 69.9; 3.8 GB
// 608 and 697.  In place counts twice too: 130 MB in place 41 us and 46-49, 200 MB 62
// and 70-72, also where the table has just been written (bf16 59 and 77, fp32 59 and
// 60).  Plain loads win there only where nothing but the clip touches one table again and
// again (200 MB: 57 for 61) and in the clip right after the norm of fp32 (100 for 107);
// non-temporal ones would win from 100 MB in place on already (32 for 34-36).
bool streams(const zero_tensor_plan* p) { return p->bytes > int64_t(256) << 20; }

int clip_impl(const zero_tensor_plan* plan, const void* table, float max_norm,
              const zero_step_result* res, const float* norms, hipStream_t stream) {
    const auto kernel = streams(plan) ? tensor_clip_kernel<true> : tensor_clip_kernel<false>;
    return in_launches(plan->n_pieces, [&](int64_t b, int64_t grid) {
        return launch(kernel, grid, lds_for_blocks(kClipBlocksPerCU), stream, pieces_of(plan, table) + b,
                      dsts_of(plan, table) + b, max_norm, res, norms);
    });
}

template <int KIND>
int clip_norm_impl(const zero_tensor_plan* plan, const void* table, float max_norm, float inv_scale,
                   const zero_step_control* ctl, zero_step_result* res, float* norms,
                   int32_t per_tensor, double* part, hipStream_t stream) {
    if (one_block_clip(plan, norms))
        return one_block_impl<KIND, true>(plan, table, max_norm, per_tensor, inv_scale, ctl, 0, res,
                                          norms, stream);
    const int64_t n = plan->n_runs + plan->n_rests;
    if (!norms && n <= kJoinPartials) {
        const int rc = partials_impl<KIND>(plan, table, part, stream);
        if (rc != ZERO_OK) return rc;
        return launch(tensor_join_clip_kernel<KIND>, plan->n_pieces, 0, stream, pieces_of(plan, table),
                      dsts_of(plan, table), max_norm, part, (int)n, inv_scale, ctl, res);
    }
    const int rc = norm_impl<KIND>(plan, table, inv_scale, ctl, 0, res, norms, part, stream);
    if (rc != ZERO_OK) return rc;
    return clip_impl(plan, table, max_norm, res, per_tensor ? norms : nullptr, stream);
}

// Resident blocks per CU of an accumulation (us; 9.4e8 elements unless said).  Added to
// what is there, two streams in and one out:
//   bf16 into fp32              1445 at 2, 1486 at 3, 1517 at 4, 1569 at 8
//   5.1e8, 1.7e8 of them         704 and 230 at 2, 714 and 230 at 3
//   with the norm               1500 at 2, 1455 at 3 (fp32 into fp32: 1749, 1793)
//   bf16 into bf16               973 at 2, 838 at 3, 874 at 4, 932 at 8
// One stream less (overwrite), the norm's squares in 64 bits and the rounding to 16 bits
// leave a block less time in which its loads are under way, and take more blocks:
//   bf16 into bf16, the norm     952 at 3, 852 at 4, 859 at 5, 928 at 8 (fp32 into bf16:
//                               1170, 1154, 1214, 1244)
//   overwrite                    668 at 3, 573 at 5, 600 at 8
//   overwrite, the norm          890 at 3, 623 at 5, 595 at 8
//   bf16 into fp32, both         913 at 3, 898 at 4, 894 at 5, 933 at 8
int add_blocks(const zero_tensor_plan* p, bool overwrite, bool norm) {
    if (overwrite && norm) return p->fp32_out ? 4 : 8;
    if (!p->fp32_out && (overwrite || norm)) return overwrite ? 5 : 4;
    return p->fp32_out && p->bytes > int64_t(2) << 30 ? 2 : 3;
}

template <int KIND>
int accumulate_impl(const zero_tensor_plan* plan, const void* table, float weight,
                    int32_t overwrite, double* part, hipStream_t stream) {
    const auto kernel = overwrite ? tensor_accumulate_kernel<KIND, true>
                                  : tensor_accumulate_kernel<KIND, false>;
    const unsigned lds = lds_for_blocks(add_blocks(plan, overwrite != 0, KIND != 0));
    return in_launches(plan->n_pieces, [&](int64_t b, int64_t grid) {
        return launch(kernel, grid, lds, stream, pieces_of(plan, table) + b,
                      dsts_of(plan, table) + b, weight, KIND ? part + b : part);
    });
}

template <int KIND>
int accumulate_norm_impl(const zero_tensor_plan* plan, const void* table, float weight,
                         int32_t overwrite, float inv_scale, const zero_step_control* ctl,
                         int32_t accumulate, zero_step_result* res, float* norms, double* part,
                         hipStream_t stream) {
    const int rc = accumulate_impl<KIND>(plan, table, weight, overwrite, part, stream);
    if (rc != ZERO_OK) return rc;
    return finish<KIND>(plan->n_pieces, plan->largest, first_pieces_of(plan, table), nullptr,
                        plan->n_tensors, inv_scale, ctl, accumulate, res, norms, part, stream);
}

}  // namespace

extern "C" {

int zero_tensor_plan_init(const zero_tensor_entry* entries, int64_t n_tensors,
                          zero_tensor_plan* plan) {
    if (!plan || n_tensors < 0 || (n_tensors > 0 && !entries)) return ZERO_EINVAL;
    if (n_tensors >= kMaxTensors) return ZERO_ERANGE;
    return plan_of(entries, n_tensors, plan);
}

int zero_tensor_plan_head(const zero_tensor_entry* entries, const zero_tensor_plan* plan,
                          void* head) {
    if (!plan || !head || plan->n_tensors < 0 || (plan->n_tensors > 0 && !entries)) return ZERO_EINVAL;
    zero_tensor_plan again;
    if (plan->n_tensors >= kMaxTensors) return ZERO_EINVAL;
    const int rc = plan_of(entries, plan->n_tensors, &again);
    if (rc != ZERO_OK) return rc;
    // whole: equal counts alone would let a plan that may be written through stand
    // for entries whose outputs overlap
    static_assert(sizeof(zero_tensor_plan) == 80, "no padding");
    if (memcmp(&again, plan, sizeof again) != 0) return ZERO_EINVAL;
    const int64_t n = plan->n_tensors;
    memset(head, 0, (size_t)plan->head_bytes);
    if (n > 0) memcpy(head, entries, (size_t)n * sizeof(zero_tensor_entry));
    int64_t* first_run = (int64_t*)first_runs_of(plan, head);
    int64_t* first_rest = (int64_t*)first_rests_of(plan, head);
    int64_t* first_piece_at = (int64_t*)first_pieces_of(plan, head);
    int64_t run = 0, rest = plan->n_runs, piece = 0;
    for (int64_t k = 0;; ++k) {
        first_run[k] = run;
        first_rest[k] = rest;
        first_piece_at[k] = piece;
        if (k == n) return ZERO_OK;
        run += runs_in(entries[k]);
        rest += rests_in(entries[k]);
        piece += pieces_in(entries[k]);
    }
}

int zero_tensor_plan_expand(const zero_tensor_plan* plan, void* table, hipStream_t stream) {
    if (!valid_plan(plan, table)) return ZERO_EINVAL;
    const int64_t units = plan->n_runs + plan->n_rests + plan->n_pieces;
    return in_launches((units + kThreads - 1) / kThreads, [&](int64_t b, int64_t grid) {
        return launch(tensor_expand_kernel, grid, 0, stream, entries_of(table),
                      first_runs_of(plan, table), first_rests_of(plan, table),
                      first_pieces_of(plan, table), plan->n_tensors, plan->n_runs, plan->n_rests,
                      plan->n_pieces, b, (Piece*)runs_of(plan, table), (Piece*)pieces_of(plan, table),
                      (void**)dsts_of(plan, table));
    });
}

size_t zero_tensor_workspace_bytes(const zero_tensor_plan* plan) {
    if (!plan || plan->n_pieces < 0 || plan->n_pieces > kMaxPieces) return 0;
    // a tensor has at least as many pieces as runs and rests
    const int64_t n = plan->n_pieces;
    return (size_t)std::max<int64_t>(2, n + fold_blocks(n)) * sizeof(double);
}

int zero_tensor_norm(const zero_tensor_plan* plan, const void* table, int32_t kind,
                     float inv_scale, const zero_step_control* ctl, zero_step_result* res,
                     float* norms, void* workspace, size_t workspace_bytes, int32_t accumulate,
                     hipStream_t stream) {
    const int rc = norm_args(plan, table, kind, inv_scale, ctl, res, workspace, workspace_bytes);
    if (rc != ZERO_OK) return rc;
    double* part = (double*)workspace;
    return kind == ZERO_NORM_L2
               ? norm_impl<ZERO_NORM_L2>(plan, table, inv_scale, ctl, accumulate, res, norms, part, stream)
               : norm_impl<ZERO_NORM_MAX>(plan, table, inv_scale, ctl, accumulate, res, norms, part, stream);
}

int zero_tensor_clip(const zero_tensor_plan* plan, const void* table, float max_norm,
                     const zero_step_result* res, const float* norms, hipStream_t stream) {
    if (!valid_plan(plan, table) || !plan->writable || !res || max_norm != max_norm)
        return ZERO_EINVAL;
    return clip_impl(plan, table, max_norm, res, norms, stream);
}

int zero_tensor_clip_norm(const zero_tensor_plan* plan, const void* table, int32_t kind,
                          float max_norm, float inv_scale, const zero_step_control* ctl,
                          zero_step_result* res, float* norms, int32_t per_tensor, void* workspace,
                          size_t workspace_bytes, hipStream_t stream) {
    if (!valid_plan(plan, table) || !plan->writable || max_norm != max_norm ||
        (per_tensor && !norms && plan->n_tensors > 0))
        return ZERO_EINVAL;
    const int rc = norm_args(plan, table, kind, inv_scale, ctl, res, workspace, workspace_bytes);
    if (rc != ZERO_OK) return rc;
    double* part = (double*)workspace;
    return kind == ZERO_NORM_L2
               ? clip_norm_impl<ZERO_NORM_L2>(plan, table, max_norm, inv_scale, ctl, res, norms,
                                              per_tensor, part, stream)
               : clip_norm_impl<ZERO_NORM_MAX>(plan, table, max_norm, inv_scale, ctl, res, norms,
                                               per_tensor, part, stream);
}

int zero_tensor_accumulate(const zero_tensor_plan* plan, const void* table, float weight,
                           int32_t overwrite, hipStream_t stream) {
    if (!valid_plan(plan, table) || !plan->writable || !__builtin_isfinite(weight)) return ZERO_EINVAL;
    return accumulate_impl<0>(plan, table, weight, overwrite, nullptr, stream);
}

int zero_tensor_accumulate_norm(const zero_tensor_plan* plan, const void* table, float weight,
                                int32_t overwrite, int32_t kind, float inv_scale,
                                const zero_step_control* ctl, zero_step_result* res, float* norms,
                                void* workspace, size_t workspace_bytes, int32_t accumulate,
                                hipStream_t stream) {
    const int rc = norm_args(plan, table, kind, inv_scale, ctl, res, workspace, workspace_bytes);
    if (rc != ZERO_OK) return rc;
    if (!plan->writable || !__builtin_isfinite(weight)) return ZERO_EINVAL;
    double* part = (double*)workspace;
    return kind == ZERO_NORM_L2
               ? accumulate_norm_impl<ZERO_NORM_L2>(plan, table, weight, overwrite, inv_scale, ctl,
                                                    accumulate, res, norms, part, stream)
               : accumulate_norm_impl<ZERO_NORM_MAX>(plan, table, weight, overwrite, inv_scale, ctl,
                                                     accumulate, res, norms, part, stream);
}

}  // extern "C"
