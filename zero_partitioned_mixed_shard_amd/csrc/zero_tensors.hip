// zero_tensors.hip -- operators over a table of gradient tensors (the
// zero_tensor_* calls of include/zero_shard.h): the norm of all of them and of
// each, clipping by it, and accumulation of one table into another.
//
// A host-built plan cuts every tensor into chunks of at most plan->chunk
// elements and the device table holds one 32-byte record per chunk, so a block
// learns all about its work from one scalar load (no search from a block
// number to a tensor) and no block spans two tensors: a chunk's partial
// belongs to one tensor, and a tensor's norm is the sum of its chunks'.
//
// Every kernel is a streaming pass bound by HBM (at most 4 operations per
// element).  Tensors start at any element, so lanes use 16-byte accesses that
// are aligned to the element only, which gfx950 global memory takes as they
// are; only a chunk's last tile, where it is short, goes element by element.
//
// Numerics: the squares and their sums are fp64 (the square of an fp32 value
// is exact there, and the sum cannot overflow), the unscale factor is applied
// to the sum; products and sums of the other calls are fp32, rounded to the
// output's type once.  Sums are folded in a fixed order: the same plan gives
// the same bits every time.

#include <math.h>

#include <algorithm>
#include <new>
#include <vector>

#include "zero_common.h"

namespace {

// One chunk of the device table.
struct Chunk {
    const void* src;
    void* dst;
    int32_t count;     // elements, 1 .. plan->chunk
    int32_t tensor;    // index in the table
    int32_t src_dtype, dst_dtype;
};
static_assert(sizeof(Chunk) == 32, "one scalar load");

// Elements per chunk.
constexpr int64_t kChunk = 16384;

// Tensor pointers come out of the table; these types make the accesses global
// ones (not flat), of 16 bytes at any element.
typedef __attribute__((address_space(1))) const char g_cbyte;
typedef __attribute__((address_space(1))) char g_byte;
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef __attribute__((address_space(1))) const u32x4_a2 g_cu32x4_a2;
typedef __attribute__((address_space(1))) u32x4_a2 g_u32x4_a2;
typedef __attribute__((address_space(1))) const uint16_t g_cu16;
typedef __attribute__((address_space(1))) uint16_t g_u16;
typedef __attribute__((address_space(1))) const float g_cf32;
typedef __attribute__((address_space(1))) float g_f32;

template <int DT>
constexpr int kBytes = DT == ZERO_FP32 ? 4 : 2;

// ---------------------------------------------------------- 8 elements -----
__device__ __forceinline__ float half_to_f32(uint16_t b) {
    return (float)__builtin_bit_cast(_Float16, b);
}
__device__ __forceinline__ float bf_to_f32(uint16_t b) {
    return __uint_as_float((uint32_t)b << 16);
}
template <int DT>
__device__ __forceinline__ float widen(uint16_t b) {
    return DT == ZERO_FP16 ? half_to_f32(b) : bf_to_f32(b);
}
// Nearest, ties to even; overflow gives inf, NaN stays (quiet) NaN.
template <int DT>
__device__ __forceinline__ uint16_t narrow(float f) {
    if (DT == ZERO_FP16) return __builtin_bit_cast(uint16_t, (_Float16)f);
    const uint32_t u = __float_as_uint(f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((u >> 16) | 0x0040u);
    return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}

// A tile of kVec elements as it lies in memory.
template <int DT>
struct Raw {
    u32x4 w[DT == ZERO_FP32 ? 2 : 1];
    __device__ __forceinline__ float get(int k) const {
        if (DT == ZERO_FP32) return __uint_as_float(w[k >> 2][k & 3]);
        return widen<DT>(half_of(w[0], k));
    }
};
template <int DT>
__device__ __forceinline__ Raw<DT> load_tile(const void* p, int e) {
    Raw<DT> r;
    g_cu32x4_a2* q = (g_cu32x4_a2*)((g_cbyte*)p + (int64_t)e * kBytes<DT>);
    r.w[0] = q[0];
    if (DT == ZERO_FP32) r.w[DT == ZERO_FP32 ? 1 : 0] = q[1];
    return r;
}
template <int DT>
__device__ __forceinline__ void store_tile(void* p, int e, const float (&v)[kVec]) {
    g_u32x4_a2* q = (g_u32x4_a2*)((g_byte*)p + (int64_t)e * kBytes<DT>);
    if (DT == ZERO_FP32) {
        u32x4 a, b;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            a[k] = __float_as_uint(v[k]);
            b[k] = __float_as_uint(v[k + 4]);
        }
        q[0] = a;
        q[1] = b;
    } else {
        uint16_t h[kVec];
#pragma unroll
        for (int k = 0; k < kVec; ++k) h[k] = narrow<DT>(v[k]);
        q[0] = pack8(h);
    }
}
template <int DT>
__device__ __forceinline__ float load_one(const void* p, int e) {
    if (DT == ZERO_FP32) return ((g_cf32*)p)[e];
    return widen<DT>(((g_cu16*)p)[e]);
}
template <int DT>
__device__ __forceinline__ void store_one(void* p, int e, float v) {
    if (DT == ZERO_FP32) ((g_f32*)p)[e] = v;
    else ((g_u16*)p)[e] = narrow<DT>(v);
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

// The block's lanes joined, in a fixed order; valid in thread 0.
template <int KIND>
__device__ __forceinline__ double block_join(double v) {
    __shared__ double part[kThreads / 64];
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v = join<KIND>(v, __shfl_xor(v, off, 64));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        v = part[0];
#pragma unroll
        for (int k = 1; k < kThreads / 64; ++k) v = join<KIND>(v, part[k]);
    }
    return v;
}

template <int KIND, int DT>
__device__ __forceinline__ double chunk_norm(const void* src, int count) {
    Norm<KIND> n;
    int e = threadIdx.x * kVec;
#pragma unroll 4
    for (; e + kVec <= count; e += kTile) {
        const Raw<DT> r = load_tile<DT>(src, e);
#pragma unroll
        for (int k = 0; k < kVec; ++k) n.add(r.get(k));
    }
    for (int end = e + kVec; e < end && e < count; ++e) n.add(load_one<DT>(src, e));
    return n.value();
}

// One partial per chunk.
template <int KIND>
__global__ void __launch_bounds__(kThreads)
tensor_norm_kernel(const Chunk* __restrict__ chunks, double* __restrict__ part) {
    const Chunk c = chunks[blockIdx.x];
    double v;
    if (c.src_dtype == ZERO_FP32) v = chunk_norm<KIND, ZERO_FP32>(c.src, c.count);
    else if (c.src_dtype == ZERO_FP16) v = chunk_norm<KIND, ZERO_FP16>(c.src, c.count);
    else v = chunk_norm<KIND, ZERO_BF16>(c.src, c.count);
    v = block_join<KIND>(v);
    if (threadIdx.x == 0) part[blockIdx.x] = v;
}

// Block b joins partials [b*kFold, (b+1)*kFold).
template <int KIND>
__global__ void __launch_bounds__(kThreads)
tensor_fold_kernel(const double* __restrict__ part, int64_t n, double* __restrict__ out) {
    double v = 0.0;
    const int64_t base = (int64_t)blockIdx.x * kFold;
#pragma unroll
    for (int k = 0; k < kFold / kThreads; ++k) {
        const int64_t j = base + k * kThreads + threadIdx.x;
        if (j < n) v = join<KIND>(v, part[j]);
    }
    v = block_join<KIND>(v);
    if (threadIdx.x == 0) out[blockIdx.x] = v;
}

// Block 0 joins the n (folded) partials into *res; block 1 + k joins tensor
// k's chunk partials into norms[k].
template <int KIND>
__global__ void __launch_bounds__(kThreads)
tensor_finish_kernel(const double* __restrict__ part, int64_t n, const double* __restrict__ chunk_part,
                     const int64_t* __restrict__ first, float inv_scale,
                     const zero_step_control* __restrict__ ctl, int accumulate,
                     zero_step_result* res, float* __restrict__ norms) {
    const float inv = ctl ? ctl->inv_scale : inv_scale;
    double v = 0.0;
    if (blockIdx.x == 0) {
        for (int64_t j = threadIdx.x; j < n; j += kThreads) v = join<KIND>(v, part[j]);
        v = block_join<KIND>(v);
        if (threadIdx.x != 0) return;
        const double x = KIND == ZERO_NORM_L2 ? v : v * v;
        uint32_t bad = x < INFINITY ? 0u : 1u;        // NaN and inf are not
        double sumsq = x * ((double)inv * (double)inv);
        if (accumulate) {
            bad |= res->overflow;
            sumsq = join<KIND>(res->sumsq, sumsq);
        }
        res->sumsq = sumsq;
        res->overflow = bad;
        res->inv_scale = inv;
        return;
    }
    const int64_t t = (int64_t)blockIdx.x - 1;
    for (int64_t j = first[t] + threadIdx.x; j < first[t + 1]; j += kThreads)
        v = join<KIND>(v, chunk_part[j]);
    v = block_join<KIND>(v);
    if (threadIdx.x == 0)
        norms[t] = (float)((KIND == ZERO_NORM_L2 ? sqrt(v) : v) * (double)inv);
}

// ------------------------------------------------------------- clip --------
// max_norm / (norm + 1e-6) where that is below 1, else 1, times the unscale
// factor; fp64, rounded once.
__device__ __forceinline__ float clip_factor(float max_norm, double norm, float inv) {
    double c = 1.0;
    if (max_norm > 0.0f) {
        const double q = (double)max_norm / (norm + 1e-6);
        if (q < 1.0) c = q;
    }
    return (float)(c * (double)inv);
}

template <int SRC, int DST>
__device__ __forceinline__ void chunk_scale(const void* src, void* dst, int count, float f) {
    int e = threadIdx.x * kVec;
#pragma unroll 4
    for (; e + kVec <= count; e += kTile) {
        const Raw<SRC> r = load_tile<SRC>(src, e);
        float v[kVec];
#pragma unroll
        for (int k = 0; k < kVec; ++k) v[k] = r.get(k) * f;
        store_tile<DST>(dst, e, v);
    }
    for (int end = e + kVec; e < end && e < count; ++e)
        store_one<DST>(dst, e, load_one<SRC>(src, e) * f);
}

// Calls go(SRC, DST as integral constants) for a chunk's types.
template <int V>
struct Int {
    static constexpr int value = V;
};
template <typename F>
__device__ __forceinline__ void by_types(const Chunk& c, F&& go) {
    auto by_dst = [&](auto src) {
        if (c.dst_dtype == ZERO_FP32) go(src, Int<ZERO_FP32>{});
        else if (c.dst_dtype == ZERO_FP16) go(src, Int<ZERO_FP16>{});
        else go(src, Int<ZERO_BF16>{});
    };
    if (c.src_dtype == ZERO_FP32) by_dst(Int<ZERO_FP32>{});
    else if (c.src_dtype == ZERO_FP16) by_dst(Int<ZERO_FP16>{});
    else by_dst(Int<ZERO_BF16>{});
}

__global__ void __launch_bounds__(kThreads)
tensor_clip_kernel(const Chunk* __restrict__ chunks, float max_norm,
                   const zero_step_result* __restrict__ res, const float* __restrict__ norms) {
    if (res->overflow) return;                       // skipped step: write nothing
    const Chunk c = chunks[blockIdx.x];
    const double norm = norms ? (double)norms[c.tensor] : sqrt(res->sumsq);
    const float f = clip_factor(max_norm, norm, res->inv_scale);
    by_types(c, [&](auto s, auto d) {
        chunk_scale<decltype(s)::value, decltype(d)::value>(c.src, c.dst, c.count, f);
    });
}

// ------------------------------------------------------- accumulate --------
// KIND 0: no norm of the result.
template <int KIND, bool FIRST, int SRC, int DST>
__device__ __forceinline__ void chunk_accumulate(const void* src, void* dst, int count, float w,
                                                 Norm<KIND>& n) {
    // the value as stored: what a later pass over dst would read
    auto stored = [](float v) { return DST == ZERO_FP32 ? v : widen<DST>(narrow<DST>(v)); };
    int e = threadIdx.x * kVec;
#pragma unroll 2
    for (; e + kVec <= count; e += kTile) {
        const Raw<SRC> x = load_tile<SRC>(src, e);
        float v[kVec];
        if (FIRST) {
#pragma unroll
            for (int k = 0; k < kVec; ++k) v[k] = w * x.get(k);
        } else {
            const Raw<DST> y = load_tile<DST>(dst, e);
#pragma unroll
            for (int k = 0; k < kVec; ++k) v[k] = fmaf(w, x.get(k), y.get(k));
        }
        if (KIND)
#pragma unroll
            for (int k = 0; k < kVec; ++k) n.add(stored(v[k]));
        store_tile<DST>(dst, e, v);
    }
    for (int end = e + kVec; e < end && e < count; ++e) {
        const float x = load_one<SRC>(src, e);
        const float v = FIRST ? w * x : fmaf(w, x, load_one<DST>(dst, e));
        if (KIND) n.add(stored(v));
        store_one<DST>(dst, e, v);
    }
}

template <int KIND, bool FIRST>
__global__ void __launch_bounds__(kThreads)
tensor_accumulate_kernel(const Chunk* __restrict__ chunks, float w, double* __restrict__ part) {
    const Chunk c = chunks[blockIdx.x];
    Norm<KIND> n;
    by_types(c, [&](auto s, auto d) {
        chunk_accumulate<KIND, FIRST, decltype(s)::value, decltype(d)::value>(c.src, c.dst, c.count,
                                                                             w, n);
    });
    if (KIND) {
        const double v = block_join<KIND>(n.value());
        if (threadIdx.x == 0) part[blockIdx.x] = v;
    }
}

// ------------------------------------------------------------- host --------
inline bool valid_table_dtype(int32_t dt) { return valid_dtype(dt) || dt == ZERO_FP32; }
inline int64_t dtype_bytes(int32_t dt) { return dt == ZERO_FP32 ? 4 : 2; }

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
    // `sorted`: disjoint spans in order; the first that ends after s begins
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
    std::sort(out.begin(), out.end(), [](const Span& a, const Span& b) { return a.begin < b.begin; });
    for (size_t k = 1; k < out.size(); ++k)
        if (out[k].begin < out[k - 1].end) return false;
    for (int64_t k = 0; k < n; ++k) {
        const zero_tensor_entry& e = entries[k];
        if (e.numel <= 0 || (e.src == e.dst && e.src_dtype == e.dst_dtype)) continue;
        if (span_of(e.src, e.numel, e.src_dtype, &s) && overlaps(out, s)) return false;
    }
    return true;
}

int plan_sizes(const zero_tensor_entry* entries, int64_t n, zero_tensor_plan* plan) {
    int64_t numel = 0, chunks = 0;
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
        if (__builtin_add_overflow(numel, e.numel, &numel)) return ZERO_ERANGE;
        chunks += (e.numel - 1) / kChunk + 1;
        if (chunks > kMaxLaunchBlocks) return ZERO_ERANGE;
    }
    plan->n_tensors = n;
    plan->numel = numel;
    plan->n_chunks = chunks;
    plan->chunk = kChunk;
    plan->table_bytes = chunks * (int64_t)sizeof(Chunk) + (n + 1) * (int64_t)sizeof(int64_t);
    plan->writable = 0;
    plan->reserved = 0;
    return ZERO_OK;
}

// What a device call needs of a plan and its table.
bool valid_plan(const zero_tensor_plan* p, const void* table) {
    return p && p->n_tensors >= 0 && p->n_tensors < kMaxLaunchBlocks && p->n_chunks >= 0 &&
           p->n_chunks <= kMaxLaunchBlocks && p->chunk > 0 && table && ((uintptr_t)table & 15) == 0;
}

inline const int64_t* first_chunks(const zero_tensor_plan* p, const void* table) {
    return (const int64_t*)((const char*)table + p->n_chunks * (int64_t)sizeof(Chunk));
}

inline int64_t folds(int64_t chunks) { return chunks <= kFinal ? 0 : (chunks + kFold - 1) / kFold; }

int norm_args(const zero_tensor_plan* plan, const void* table, int32_t kind, float inv_scale,
              const zero_step_control* ctl, const zero_step_result* res, const void* workspace,
              size_t workspace_bytes) {
    if (!valid_plan(plan, table) || (kind != ZERO_NORM_L2 && kind != ZERO_NORM_MAX)) return ZERO_EINVAL;
    if (!res || !workspace || ((uintptr_t)workspace & 7) != 0) return ZERO_EINVAL;
    if (!ctl && (!(inv_scale > 0.0f) || !__builtin_isfinite(inv_scale))) return ZERO_EINVAL;
    if (workspace_bytes < zero_tensor_workspace_bytes(plan)) return ZERO_EINVAL;
    return ZERO_OK;
}

// Joins the chunk partials at the workspace's start into *res and norms.
template <int KIND>
int finish(const zero_tensor_plan* plan, const void* table, float inv_scale,
           const zero_step_control* ctl, int32_t accumulate, zero_step_result* res, float* norms,
           double* part, hipStream_t stream) {
    const double* last = part;
    int64_t n = plan->n_chunks;
    if (const int64_t blocks = folds(n)) {
        const int rc = launch(tensor_fold_kernel<KIND>, blocks, 0, stream, part, n, part + n);
        if (rc != ZERO_OK) return rc;
        last = part + n;
        n = blocks;
    }
    return launch(tensor_finish_kernel<KIND>, 1 + (norms ? plan->n_tensors : 0), 0, stream, last, n,
                  part, first_chunks(plan, table), inv_scale, ctl, (int)(accumulate != 0), res, norms);
}

template <int KIND>
int norm_impl(const zero_tensor_plan* plan, const void* table, float inv_scale,
              const zero_step_control* ctl, int32_t accumulate, zero_step_result* res, float* norms,
              double* part, hipStream_t stream) {
    if (plan->n_chunks > 0) {
        const int rc = launch(tensor_norm_kernel<KIND>, plan->n_chunks, 0, stream,
                              (const Chunk*)table, part);
        if (rc != ZERO_OK) return rc;
    }
    return finish<KIND>(plan, table, inv_scale, ctl, accumulate, res, norms, part, stream);
}

template <int KIND>
int accumulate_impl(const zero_tensor_plan* plan, const void* table, float weight,
                    int32_t overwrite, double* part, hipStream_t stream) {
    if (plan->n_chunks == 0) return ZERO_OK;
    return overwrite ? launch(tensor_accumulate_kernel<KIND, true>, plan->n_chunks, 0, stream,
                              (const Chunk*)table, weight, part)
                     : launch(tensor_accumulate_kernel<KIND, false>, plan->n_chunks, 0, stream,
                              (const Chunk*)table, weight, part);
}

}  // namespace

extern "C" {

int zero_tensor_plan_init(const zero_tensor_entry* entries, int64_t n_tensors,
                          zero_tensor_plan* plan) {
    if (!plan || n_tensors < 0 || (n_tensors > 0 && !entries)) return ZERO_EINVAL;
    if (n_tensors >= kMaxLaunchBlocks) return ZERO_ERANGE;
    const int rc = plan_sizes(entries, n_tensors, plan);
    if (rc != ZERO_OK) return rc;
    try {
        plan->writable = writable(entries, n_tensors) ? 1 : 0;
    } catch (const std::bad_alloc&) {
        return ZERO_ENOMEM;
    }
    return ZERO_OK;
}

int zero_tensor_plan_table(const zero_tensor_entry* entries, const zero_tensor_plan* plan,
                           void* table) {
    if (!plan || !table || plan->n_tensors < 0 || (plan->n_tensors > 0 && !entries)) return ZERO_EINVAL;
    zero_tensor_plan again;
    const int rc = plan_sizes(entries, plan->n_tensors, &again);
    if (rc != ZERO_OK) return rc;
    if (again.n_chunks != plan->n_chunks || again.chunk != plan->chunk) return ZERO_EINVAL;
    Chunk* c = (Chunk*)table;
    int64_t* first = (int64_t*)((char*)table + plan->n_chunks * (int64_t)sizeof(Chunk));
    int64_t at = 0;
    for (int64_t k = 0; k < plan->n_tensors; ++k) {
        const zero_tensor_entry& e = entries[k];
        first[k] = at;
        for (int64_t b = 0; b < e.numel; b += plan->chunk) {
            Chunk& r = c[at++];
            r.src = (const char*)e.src + b * dtype_bytes(e.src_dtype);
            r.dst = (char*)e.dst + b * dtype_bytes(e.dst_dtype);
            r.count = (int32_t)std::min(plan->chunk, e.numel - b);
            r.tensor = (int32_t)k;
            r.src_dtype = e.src_dtype;
            r.dst_dtype = e.dst_dtype;
        }
    }
    first[plan->n_tensors] = at;
    return ZERO_OK;
}

size_t zero_tensor_workspace_bytes(const zero_tensor_plan* plan) {
    if (!plan || plan->n_chunks < 0) return 0;
    const size_t partials = (size_t)(plan->n_chunks + folds(plan->n_chunks));
    return std::max<size_t>(2, partials) * sizeof(double);
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
    if (plan->n_chunks == 0) return ZERO_OK;
    return launch(tensor_clip_kernel, plan->n_chunks, 0, stream, (const Chunk*)table, max_norm, res,
                  norms);
}

int zero_tensor_clip_norm(const zero_tensor_plan* plan, const void* table, int32_t kind,
                          float max_norm, float inv_scale, const zero_step_control* ctl,
                          zero_step_result* res, float* norms, int32_t per_tensor, void* workspace,
                          size_t workspace_bytes, hipStream_t stream) {
    if (!valid_plan(plan, table) || !plan->writable || max_norm != max_norm ||
        (per_tensor && !norms && plan->n_tensors > 0))
        return ZERO_EINVAL;
    const int rc = zero_tensor_norm(plan, table, kind, inv_scale, ctl, res, norms, workspace,
                                    workspace_bytes, 0, stream);
    if (rc != ZERO_OK) return rc;
    return zero_tensor_clip(plan, table, max_norm, res, per_tensor ? norms : nullptr, stream);
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
    int rc = norm_args(plan, table, kind, inv_scale, ctl, res, workspace, workspace_bytes);
    if (rc != ZERO_OK) return rc;
    if (!plan->writable || !__builtin_isfinite(weight)) return ZERO_EINVAL;
    double* part = (double*)workspace;
    if (kind == ZERO_NORM_L2) {
        rc = accumulate_impl<ZERO_NORM_L2>(plan, table, weight, overwrite, part, stream);
        if (rc != ZERO_OK) return rc;
        return finish<ZERO_NORM_L2>(plan, table, inv_scale, ctl, accumulate, res, norms, part, stream);
    }
    rc = accumulate_impl<ZERO_NORM_MAX>(plan, table, weight, overwrite, part, stream);
    if (rc != ZERO_OK) return rc;
    return finish<ZERO_NORM_MAX>(plan, table, inv_scale, ctl, accumulate, res, norms, part, stream);
}

}  // extern "C"
