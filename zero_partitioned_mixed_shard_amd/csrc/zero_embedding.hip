// zero_embedding.hip -- rows of the vocabulary table by tokens: lookup with scaling
// (zero_embedding_lookup) and its gradient by sorted tokens (zero_embedding_grad), from
// and into an owner's slice of the flat table.
//
// Gradient.  dW[v] = scale * sum of dy[t] over the tokens t of v.  The tokens are sorted
// by their id, stably, so equal ones lie next to each other in the order of t.  The
// sorted list is cut into chunks; a wave adds up the rows of a chunk for 512 columns, in
// fp32, and writes the sums of the ids that begin and end in its chunk.  What an id
// has in a chunk beside others goes to the workspace, and a second pass adds these
// up in order.  No atomics on floats: the same call gives the same bits.
//
// Everything here is bound by HBM (dy is read once, rows that tokens have are read and
// written once) or, for few tokens, by the launches.

#include <math.h>

#include "zero_common.h"

namespace {

typedef u32x4 u32x4_a2 __attribute__((aligned(2)));

constexpr int kCols = 8;                   // columns of a lane
constexpr int kSlab = 64 * kCols;          // columns of a wave
constexpr int kSortLanes = 1024, kSortWaves = kSortLanes / 64;
constexpr int kSmallSort = 8192;           // tokens that one block sorts in LDS
constexpr int kBigLanes = 512, kBigWaves = kBigLanes / 64;
constexpr int kSortTile = 2048;            // tokens of a block of the larger sort
// Tokens of a chunk, and (chunk, 512 columns) units that are enough for the device: the
// gradient of 16384 tokens of 4096 takes 115 us with 4096 units and 119 with 8192 (more
// parts to join).
constexpr int64_t kLeastChunk = 8, kMostChunk = 512, kChunkUnits = 4096;
// Bytes that a wave clears, about.
constexpr int64_t kClearBytes = 32768;
// (A pass over 16384 to 65537 tokens takes 4 to 5 us for the counts and 7 to 8 for the
// scatter, two passes up to 2^18 ids: launches and chains of dependent accesses, not bytes.)
// Blocks whose counts each block of the larger sort adds up by itself; more take a launch.
constexpr int64_t kFewBlocks = 64;
constexpr int kDigit = 9, kBins = 1 << kDigit;   // most bits of a pass

template <int DT>
constexpr int kSize = DT == ZERO_FP32 ? 4 : 2;

template <int DT>
__device__ __forceinline__ float widen(uint16_t b) {
    return DT == ZERO_FP16 ? (float)__builtin_bit_cast(_Float16, b) : __uint_as_float((uint32_t)b << 16);
}
// Nearest, ties to even; overflow gives inf, NaN stays (quiet) NaN.
template <int DT>
__device__ __forceinline__ uint16_t narrow(float f) {
    asm("" : "+v"(f));      // rounded to fp32 before (the compiler would skip that)
    if (DT == ZERO_FP16) return __builtin_bit_cast(uint16_t, (_Float16)f);
    const uint32_t u = __float_as_uint(f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((u >> 16) | 0x0040u);
    return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}

// 8 consecutive elements as they lie in memory, which may begin at any element.
template <int DT>
struct Raw8 {
    static constexpr int kQuads = kSize<DT> / 2;
    u32x4 q[kQuads];
    __device__ __forceinline__ float get(int k) const {
        if constexpr (DT == ZERO_FP32) return __uint_as_float(q[k >> 2][k & 3]);
        else return widen<DT>(half_of(q[0], k));
    }
};
template <int DT, bool NT>
__device__ __forceinline__ Raw8<DT> load8(const void* base, int64_t e) {
    Raw8<DT> r;
    const char* p = (const char*)base + e * kSize<DT>;
#pragma unroll
    for (int k = 0; k < Raw8<DT>::kQuads; ++k) {
        const u32x4_a2* c = (const u32x4_a2*)p + k;
        r.q[k] = NT ? __builtin_nontemporal_load(c) : *c;
    }
    return r;
}
template <int DT, bool NT>
__device__ __forceinline__ void store8(void* base, int64_t e, const float* v) {
    char* p = (char*)base + e * kSize<DT>;
#pragma unroll
    for (int k = 0; k < Raw8<DT>::kQuads; ++k) {
        u32x4 w;
        if constexpr (DT == ZERO_FP32) {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = __float_as_uint(v[4 * k + j]);
        } else {
            uint16_t h[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) h[j] = narrow<DT>(v[j]);
            w = pack8(h);
        }
        u32x4_a2* c = (u32x4_a2*)p + k;
        if (NT) __builtin_nontemporal_store(w, c);
        else *c = w;
    }
}
template <int DT>
__device__ __forceinline__ float load1(const void* base, int64_t e) {
    if constexpr (DT == ZERO_FP32) return ((const float*)base)[e];
    else return widen<DT>(((const uint16_t*)base)[e]);
}
template <int DT>
__device__ __forceinline__ void store1(void* base, int64_t e, float v) {
    if constexpr (DT == ZERO_FP32) ((float*)base)[e] = v;
    else ((uint16_t*)base)[e] = narrow<DT>(v);
}

// The table's slice: elements [begin, begin + count) of vocab * dim.
struct Slice {
    int64_t vocab, dim, begin, count;
};
__device__ __forceinline__ int64_t id_at(const void* ids, int wide, int64_t t) {
    return wide ? ((const int64_t*)ids)[t] : (int64_t)((const int32_t*)ids)[t];
}

// ------------------------------------------------------------ lookup -------
// A wave takes 1024 columns of a token, 16 of each lane in two runs of 8.  16384 tokens of
// 4096 bf16 into fp32 took 68 us (512 columns the same, 2048 79), 4.6 TB/s; stored
// non-temporally 106, since a lane's 32 bytes go in two stores that each fill half of
// every line.  16-bit results, whose stores fill lines, gain 10-15 % by it.
template <int DT>
constexpr bool kNtOut = DT != ZERO_FP32;
constexpr int kLookupRuns = 2, kLookupCols = kSlab * kLookupRuns;

template <int SRC, int DST>
__global__ void __launch_bounds__(kThreads)
embedding_lookup_kernel(void* __restrict__ out, int64_t out_ld, const void* __restrict__ ids, int wide,
                        int64_t n_tokens, uint32_t parts, const void* __restrict__ table, Slice s, float scale,
                        int64_t blk0) {
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t u = (blk0 + blockIdx.x) * (kThreads / 64) + w;
    const int64_t token = u >> 32 ? u / parts : (int64_t)((uint32_t)u / parts);
    if (token >= n_tokens) return;
    const int64_t id = id_at(ids, wide, token);
    const bool known = id >= 0 && id < s.vocab;
    const int64_t first = (u - token * parts) * kLookupCols + (threadIdx.x & 63) * kCols;
    const int64_t row = known ? id * s.dim - s.begin : 0;
    Raw8<SRC> r[kLookupRuns];
    bool whole[kLookupRuns];
#pragma unroll
    for (int q = 0; q < kLookupRuns; ++q) {
        const int64_t col = first + q * kSlab, at = row + col;
        whole[q] = known && col + kCols <= s.dim && at >= 0 && at + kCols <= s.count;
        if (whole[q]) r[q] = load8<SRC, false>(table, at);
    }
#pragma unroll
    for (int q = 0; q < kLookupRuns; ++q) {
        const int64_t col = first + q * kSlab, at = row + col, to = token * out_ld + col;
        if (col >= s.dim) continue;
        const int n = (int)(s.dim - col < kCols ? s.dim - col : kCols);
        float v[kCols];
        if (whole[q]) {
#pragma unroll
            for (int k = 0; k < kCols; ++k) v[k] = scale * r[q].get(k);
        } else {
#pragma unroll
            for (int k = 0; k < kCols; ++k) {
                const int64_t e = at + k;
                v[k] = known && k < n && e >= 0 && e < s.count ? scale * load1<SRC>(table, e) : 0.0f;
            }
        }
        if (n == kCols) {
            store8<DST, kNtOut<DST>>(out, to, v);
        } else {
#pragma unroll
            for (int k = 0; k < kCols; ++k)
                if (k < n) store1<DST>(out, to + k, v[k]);
        }
    }
}

// ------------------------------------------------------------ sort ---------
// The key of a token: its id, or `vocab`, after all ids, where it gives nothing to the
// slice (an id that is none, the padding id, a row outside).
struct Keys {
    const void* ids;
    int wide;
    int64_t n, padding;
    Slice s;
    __device__ __forceinline__ uint32_t get(int64_t t) const {
        const int64_t id = id_at(ids, wide, t);
        if (id < 0 || id >= s.vocab || id == padding) return (uint32_t)s.vocab;
        const int64_t a = id * s.dim - s.begin;
        return a + s.dim <= 0 || a >= s.count ? (uint32_t)s.vocab : (uint32_t)id;
    }
};

// Stable ranks of a wave's keys, 64 at a time: how many equal digits are before each
// in the wave, counted on in count[digit].
__device__ __forceinline__ int wave_rank(uint32_t digit, bool valid, int bits, uint32_t* count, int lane) {
    uint64_t peers = __ballot(valid);
    for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot((digit >> b) & 1);
        peers &= (digit >> b) & 1 ? set : ~set;
    }
    const int below = __popcll(peers & ((uint64_t(1) << lane) - 1));
    const uint32_t before = valid ? count[digit] : 0;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (valid && below == 0) count[digit] = before + (uint32_t)__popcll(peers);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    return (int)before + below;
}

// count[wave][bin] into the number of keys before the wave's first of that bin; add[bin]
// (or the bins' own sums) is where a bin begins.  Lanes 0 to 511 take a bin each.
template <int WAVES>
__device__ __forceinline__ void bin_starts(uint32_t (*count)[kBins], const uint32_t* start, uint32_t* sums) {
    const int t = threadIdx.x;
    uint32_t total = 0;
    if (t < kBins)
        for (int w = 0; w < WAVES; ++w) {
            const uint32_t c = count[w][t];
            count[w][t] = total;
            total += c;
        }
    uint32_t base = 0;
    if (start == nullptr) {
        // exclusive sum over the bins: within waves, then over the 8 waves that hold them
        uint32_t v = total;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const uint32_t o = (uint32_t)__shfl_up((int)v, off, 64);
            if ((t & 63) >= off) v += o;
        }
        if (t < kBins && (t & 63) == 63) sums[t >> 6] = v;
        __syncthreads();
        base = v - total;
        if (t < kBins)
            for (int w = 0; w < (t >> 6); ++w) base += sums[w];
    } else if (t < kBins) {
        base = start[t];
    }
    if (t < kBins)
        for (int w = 0; w < WAVES; ++w) count[w][t] += base;
    __syncthreads();
}

// Up to kSmallSort tokens by one block in LDS.
__global__ void __launch_bounds__(kSortLanes)
embedding_sort_small_kernel(Keys keys, int passes, int bits, uint32_t* __restrict__ out_key,
                            uint32_t* __restrict__ out_pos, uint32_t* __restrict__ n_valid) {
    __shared__ uint32_t count[kSortWaves][kBins];
    __shared__ uint32_t sums[kSortWaves];
    __shared__ uint32_t lk[kSmallSort], lp[kSmallSort];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, n = (int)keys.n;
    constexpr int kRounds = kSmallSort / kSortLanes;
    const int rounds = (n + kSortLanes - 1) / kSortLanes;    // of every wave
    uint32_t k[kRounds], p[kRounds];
    int rank[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const int t = (w * rounds + r) * 64 + lane;
        k[r] = r < rounds && t < n ? keys.get(t) : 0;
        p[r] = (uint32_t)t;
    }
    for (int pass = 0; pass < passes; ++pass) {
        for (int b = lane; b < kBins; b += 64) count[w][b] = 0;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            if (r >= rounds) break;
            const bool valid = (w * rounds + r) * 64 + lane < n;
            rank[r] = wave_rank((k[r] >> (pass * bits)) & ((1u << bits) - 1), valid, bits, count[w], lane);
        }
        __syncthreads();
        bin_starts<kSortWaves>(count, nullptr, sums);
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            if (r >= rounds) break;
            if ((w * rounds + r) * 64 + lane < n) {
                const uint32_t at = count[w][(k[r] >> (pass * bits)) & ((1u << bits) - 1)] + (uint32_t)rank[r];
                lk[at] = k[r];
                lp[at] = p[r];
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int t = (w * rounds + r) * 64 + lane;
            if (r < rounds && t < n) {
                k[r] = lk[t];
                p[r] = lp[t];
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const int t = (w * rounds + r) * 64 + lane;
        if (r < rounds && t < n) {
            out_key[t] = k[r];
            out_pos[t] = p[r];
            // the first of no row, or the end
            if (k[r] == (uint32_t)keys.s.vocab && (t == 0 || lk[t - 1] != k[r])) *n_valid = (uint32_t)t;
            if (t + 1 == n && k[r] != (uint32_t)keys.s.vocab) *n_valid = (uint32_t)n;
        }
    }
}

// A pass of the larger sort reads (key, position) pairs, or the ids in the first.
struct Pairs {
    const uint32_t *key, *pos;
};
__device__ __forceinline__ uint32_t key_of(const Keys& keys, const Pairs& in, int64_t t) {
    return in.key ? in.key[t] : keys.get(t);
}
__global__ void __launch_bounds__(kBigLanes)
embedding_count_kernel(Keys keys, Pairs in, int shift, int bits, int64_t blocks, uint32_t* __restrict__ counts) {
    __shared__ uint32_t bin[kBins];
    if (threadIdx.x < kBins) bin[threadIdx.x] = 0;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * kSortTile;
#pragma unroll
    for (int r = 0; r < kSortTile / kBigLanes; ++r) {
        const int64_t t = t0 + r * kBigLanes + threadIdx.x;
        if (t < keys.n) atomicAdd(&bin[(key_of(keys, in, t) >> shift) & ((1u << bits) - 1)], 1u);
    }
    __syncthreads();
    if (threadIdx.x < (1u << bits)) counts[(int64_t)threadIdx.x * blocks + blockIdx.x] = bin[threadIdx.x];
}
// Exclusive sums of n counts, by one block.
__global__ void __launch_bounds__(kSortLanes)
embedding_scan_kernel(uint32_t* __restrict__ counts, int64_t n) {
    __shared__ uint32_t sums[kSortWaves];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    uint32_t carry = 0;
    for (int64_t at = 0; at < n; at += kSortLanes * 4) {
        uint32_t c[4], total = 0;
        const int64_t e = at + threadIdx.x * 4;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            c[k] = e + k < n ? counts[e + k] : 0;
            total += c[k];
        }
        uint32_t v = total;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const uint32_t o = (uint32_t)__shfl_up((int)v, off, 64);
            if (lane >= off) v += o;
        }
        if (lane == 63) sums[w] = v;
        __syncthreads();
        uint32_t base = carry + v - total, all = 0;
        for (int k = 0; k < kSortWaves; ++k) {
            if (k < w) base += sums[k];
            all += sums[k];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (e + k < n) counts[e + k] = base;
            base += c[k];
        }
        carry += all;
        __syncthreads();
    }
}
__global__ void __launch_bounds__(kBigLanes)
embedding_scatter_kernel(Keys keys, Pairs in, int shift, int bits, int64_t blocks,
                         const uint32_t* __restrict__ counts, int scanned, uint32_t* __restrict__ out_key,
                         uint32_t* __restrict__ out_pos) {
    __shared__ uint32_t count[kBigWaves][kBins];
    __shared__ uint32_t start[kBins], sums[kBigWaves];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    for (int b = lane; b < kBins; b += 64) count[w][b] = 0;
    if (!scanned) {
        // the counts as they are: those of the bins before, and of the blocks before in the bin
        const uint32_t* c = counts + (int64_t)threadIdx.x * blocks;
        uint32_t all = 0, before = 0;
        if (threadIdx.x < (1u << bits)) {
#pragma unroll 8
            for (int b = 0; b < (int)blocks; ++b) {
                const uint32_t v = c[b];
                all += v;
                before += b < (int)blockIdx.x ? v : 0;
            }
        }
        uint32_t v = all;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const uint32_t o = (uint32_t)__shfl_up((int)v, off, 64);
            if (lane >= off) v += o;
        }
        if (lane == 63) sums[w] = v;
        __syncthreads();
        uint32_t base = v - all;
        for (int k = 0; k < w; ++k) base += sums[k];
        if (threadIdx.x < kBins) start[threadIdx.x] = base + before;
    } else if (threadIdx.x < kBins) {
        start[threadIdx.x] = threadIdx.x < (1u << bits) ? counts[(int64_t)threadIdx.x * blocks + blockIdx.x] : 0;
    }
    __syncthreads();
    constexpr int kRounds = kSortTile / kBigLanes;
    const int64_t t0 = (int64_t)blockIdx.x * kSortTile + w * kRounds * 64 + lane;
    uint32_t k[kRounds], p[kRounds];
    int rank[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const int64_t t = t0 + r * 64;
        k[r] = t < keys.n ? key_of(keys, in, t) : 0;
        p[r] = t < keys.n && in.key ? in.pos[t] : (uint32_t)t;
    }
#pragma unroll
    for (int r = 0; r < kRounds; ++r)
        rank[r] = wave_rank((k[r] >> shift) & ((1u << bits) - 1), t0 + r * 64 < keys.n, bits, count[w], lane);
    __syncthreads();
    bin_starts<kBigWaves>(count, start, nullptr);
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        if (t0 + r * 64 >= keys.n) continue;
        const uint32_t at = count[w][(k[r] >> shift) & ((1u << bits) - 1)] + (uint32_t)rank[r];
        out_key[at] = k[r];
        out_pos[at] = p[r];
    }
}

// ------------------------------------------------------------ sums ---------
struct Sorted {
    const uint32_t *key, *pos, *n_valid;
    int64_t most;              // chunks there is room for
    uint32_t slabs;
    float* part;               // [chunk][0: of an id that began before; 1: that goes on][dim]
    int64_t n, chunk;          // tokens with a row, and of a chunk
    // Chunks go by the tokens that have a row: an owner of a few rows has few.
    __device__ __forceinline__ void begin() {
        n = n_valid ? (int64_t)*n_valid : 0;
        chunk = kLeastChunk;
        while ((n + chunk - 1) / chunk > most) chunk *= 2;
    }
};

// Adds scale * v to row `id`, columns col .. of the slice (or stores it).
template <int DST>
__device__ __forceinline__ void emit(void* grad, const Slice& s, int64_t id, int64_t col, const float* v,
                                     float scale, int overwrite) {
    const int64_t at = id * s.dim + col - s.begin;
    const int n = (int)(s.dim - col < kCols ? s.dim - col : kCols);
    if (n <= 0) return;
    if (n == kCols && at >= 0 && at + kCols <= s.count) {
        float y[kCols];
        if (overwrite) {
#pragma unroll
            for (int k = 0; k < kCols; ++k) y[k] = scale * v[k];
        } else {
            const Raw8<DST> old = load8<DST, false>(grad, at);
#pragma unroll
            for (int k = 0; k < kCols; ++k) y[k] = fmaf(scale, v[k], old.get(k));
        }
        store8<DST, false>(grad, at, y);
        return;
    }
#pragma unroll
    for (int k = 0; k < kCols; ++k) {
        const int64_t e = at + k;
        if (k < n && e >= 0 && e < s.count)
            store1<DST>(grad, e, overwrite ? scale * v[k] : fmaf(scale, v[k], load1<DST>(grad, e)));
    }
}
__device__ __forceinline__ void store_part(float* part, int64_t dim, int64_t col, const float* v) {
    if (col + kCols <= dim) {
        store8<ZERO_FP32, false>(part, col, v);
    } else {
#pragma unroll
        for (int k = 0; k < kCols; ++k)
            if (col + k < dim) part[col + k] = v[k];
    }
}
__device__ __forceinline__ void add_part(const float* part, int64_t dim, int64_t col, float* v) {
    if (col + kCols <= dim) {
        const Raw8<ZERO_FP32> r = load8<ZERO_FP32, false>(part, col);
#pragma unroll
        for (int k = 0; k < kCols; ++k) v[k] += r.get(k);
    } else {
#pragma unroll
        for (int k = 0; k < kCols; ++k)
            if (col + k < dim) v[k] += part[col + k];
    }
}

// The first of the sorted tokens [0, n) whose key is not below `key`: 64 are looked at in a
// round, 3 rounds for 2^18 tokens.  The wave's lanes together.
__device__ __forceinline__ int64_t wave_lower_bound(const uint32_t* keys, int64_t n, int64_t key) {
    int64_t lo = 0, hi = n;
    while (lo < hi) {
        const int64_t step = (hi - lo + 63) / 64, at = lo + (int64_t)(threadIdx.x & 63) * step;
        const int c = __popcll(__ballot(at < hi && (int64_t)keys[at] < key));   // the first c are below
        if (c == 0) return lo;
        const int64_t next = lo + (int64_t)c * step;
        lo += (int64_t)(c - 1) * step + 1;
        hi = next < hi ? next : hi;
    }
    return lo;
}

// Rows of the slice that no token has become zero: the first blocks of the launch, a
// wave for `rows` rows.  Rows without tokens between two that have some are one run.
template <int DST>
__device__ __forceinline__ void clear_rows(const Sorted& q, void* grad, const Slice& s, int64_t u, int rows) {
    const int lane = threadIdx.x & 63;
    const int64_t first = s.begin / s.dim + u * rows;
    const int64_t last = (s.begin + s.count + s.dim - 1) / s.dim;
    if (first >= last) return;
    const int n = (int)(last - first < rows ? last - first : rows);
    int64_t lo = wave_lower_bound(q.key, q.n, first);
    const int64_t end = wave_lower_bound(q.key, q.n, first + n);
    bool mine = lane < n;
    if (mine) {                              // the first sorted token not before the lane's row
        const int64_t row = first + lane;
        int64_t hi = end;
        while (lo < hi) {
            const int64_t mid = (lo + hi) >> 1;
            if ((int64_t)q.key[mid] < row) lo = mid + 1;
            else hi = mid;
        }
        mine = !(lo < end && (int64_t)q.key[lo] == row);
    }
    constexpr int64_t W = 16 / kSize<DST>;
    uint64_t todo = __ballot(mine);
    while (todo) {
        const int r = __ffsll((unsigned long long)todo) - 1;
        const uint64_t rest = ~(todo >> r);
        const int run = rest ? __ffsll((unsigned long long)rest) - 1 : 64;
        todo &= r + run >= 64 ? 0 : ~uint64_t(0) << (r + run);
        int64_t a = (first + r) * s.dim - s.begin, b = a + run * s.dim;
        if (a < 0) a = 0;
        if (b > s.count) b = s.count;
        // up to 16-byte alignment, whole 16 bytes, the rest
        const int64_t skew = (int64_t)(((uintptr_t)grad / kSize<DST> + (uintptr_t)a) % W);
        int64_t head = skew ? W - skew : 0;
        if (head > b - a) head = b - a;
        const int64_t whole = (b - a - head) / W, tail = a + head + whole * W;
        if (lane < head) store1<DST>(grad, a + lane, 0.0f);
        u32x4* p = (u32x4*)((char*)grad + (a + head) * kSize<DST>);
        for (int64_t k = lane; k < whole; k += 64) __builtin_nontemporal_store(u32x4{0, 0, 0, 0}, p + k);
        if (lane < b - tail) store1<DST>(grad, tail + lane, 0.0f);
    }
}

// How many of the sorted tokens have a row: one wave.
__global__ void __launch_bounds__(64)
embedding_valid_kernel(const uint32_t* __restrict__ key, int64_t n, uint32_t none, uint32_t* __restrict__ n_valid) {
    const int64_t lo = wave_lower_bound(key, n, none);
    if (threadIdx.x == 0) *n_valid = (uint32_t)lo;
}

// A wave: a chunk's rows of dy for 512 columns, kRowsAhead at a time, with the old values of
// the rows that end among them.  16384 rows of 4096 bf16 into fp32 sums take 75 us, 4.2 TB/s,
// in the order of their ids, which is none of memory's; with 8 rows ahead the whole gradient
// takes 133 us in the place of 115.
constexpr int kRowsAhead = 4;

template <int SRC, int DST>
__global__ void __launch_bounds__(kThreads)
embedding_sum_kernel(Sorted q, const void* __restrict__ dy, int64_t dy_ld, void* __restrict__ grad, Slice s,
                     float scale, int overwrite, int64_t clear_blocks, int rows, int64_t blk0) {
    const int64_t blk = blk0 + blockIdx.x;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    q.begin();
    if (blk < clear_blocks) {
        clear_rows<DST>(q, grad, s, blk * (kThreads / 64) + w, rows);
        return;
    }
    const int64_t u = (blk - clear_blocks) * (kThreads / 64) + w;
    const int64_t c = u >> 32 ? u / q.slabs : (int64_t)((uint32_t)u / q.slabs);
    const int64_t a = c * q.chunk, b = a + q.chunk < q.n ? a + q.chunk : q.n;
    if (a >= b) return;
    const int64_t col = (u - c * q.slabs) * kSlab + (threadIdx.x & 63) * kCols;
    const bool active = col < s.dim, whole = col + kCols <= s.dim;
    float* part = q.part + 2 * c * s.dim;
    const uint32_t before = a > 0 ? q.key[a - 1] : ~0u, after = b < q.n ? q.key[b] : ~0u;
    uint32_t id = q.key[a];
    bool began = before == id;                     // in an earlier chunk
    float sum[kCols] = {0, 0, 0, 0, 0, 0, 0, 0};
    constexpr int U = kRowsAhead;
    for (int64_t i = a; i < b; i += U) {
        Raw8<SRC> r[U];
        Raw8<DST> old[U];
        uint32_t key[U + 1];
        bool has[U];
#pragma unroll
        for (int k = 0; k <= U; ++k) key[k] = i + k < b ? q.key[i + k] : after;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            has[k] = false;
            if (i + k >= b || !active) continue;
            const int64_t row = (int64_t)q.pos[i + k] * dy_ld + col;
            if (whole) {
                r[k] = load8<SRC, true>(dy, row);
            } else {
                float v[kCols];
#pragma unroll
                for (int e = 0; e < kCols; ++e) v[e] = col + e < s.dim ? load1<SRC>(dy, row + e) : 0.0f;
                if constexpr (SRC == ZERO_FP32) {
#pragma unroll
                    for (int e = 0; e < kCols; ++e) r[k].q[e >> 2][e & 3] = __float_as_uint(v[e]);
                } else {
                    uint16_t h[8];
#pragma unroll
                    for (int e = 0; e < kCols; ++e) h[e] = narrow<SRC>(v[e]);
                    r[k].q[0] = pack8(h);
                }
            }
            const int64_t at = (int64_t)key[k] * s.dim + col - s.begin;
            has[k] = !overwrite && key[k + 1] != key[k] && whole && at >= 0 && at + kCols <= s.count;
            if (has[k]) old[k] = load8<DST, false>(grad, at);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (i + k >= b) break;
            if (active) {
#pragma unroll
                for (int e = 0; e < kCols; ++e) sum[e] += r[k].get(e);
            }
            if (key[k + 1] == key[k] && i + k + 1 < b) continue;
            // the id's last token, or the chunk's
            if (active) {
                if (began) {
                    store_part(part, s.dim, col, sum);
                } else if (key[k + 1] == key[k]) {
                    store_part(part + s.dim, s.dim, col, sum);
                } else if (has[k]) {
                    float y[kCols];
#pragma unroll
                    for (int e = 0; e < kCols; ++e) y[e] = fmaf(scale, sum[e], old[k].get(e));
                    store8<DST, false>(grad, (int64_t)key[k] * s.dim + col - s.begin, y);
                } else {
                    emit<DST>(grad, s, key[k], col, sum, scale, overwrite);
                }
            }
            began = false;
#pragma unroll
            for (int e = 0; e < kCols; ++e) sum[e] = 0.0f;
        }
    }
}

// The ids that go on past a chunk's end, at the chunk where they begin: a block adds up
// their parts of the following chunks for 512 columns, its waves a quarter each, in order.
// 11 us for 16384 tokens of 4096.
template <int DST>
__global__ void __launch_bounds__(kThreads)
embedding_join_kernel(Sorted q, void* __restrict__ grad, Slice s, float scale, int overwrite, int64_t blk0) {
    __shared__ float quarter[kThreads / 64][kSlab];
    q.begin();
    const int64_t u = blk0 + blockIdx.x, c = u >> 32 ? u / q.slabs : (int64_t)((uint32_t)u / q.slabs);
    const int64_t a = c * q.chunk, b = a + q.chunk;
    if (b >= q.n) return;
    const uint32_t id = q.key[b - 1];
    if (q.key[b] != id) return;
    // the id begins in this chunk, not before
    if (q.key[a] == id && a > 0 && q.key[a - 1] == id) return;
    int64_t lo = b, hi = q.n;                      // first token after the id's
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (q.key[mid] <= id) lo = mid + 1;
        else hi = mid;
    }
    const int64_t more = (lo - 1) / q.chunk - c;   // chunks that it goes on in
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t col = (u - c * q.slabs) * kSlab + lane * kCols;
    const int64_t per = (more + 3) / 4, from = w * per, to = from + per < more ? from + per : more;
    float sum[kCols] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (col < s.dim) {
#pragma unroll 8
        for (int64_t k = from; k < to; ++k) add_part(q.part + 2 * (c + 1 + k) * s.dim, s.dim, col, sum);
    }
#pragma unroll
    for (int e = 0; e < kCols; ++e) quarter[w][lane * kCols + e] = sum[e];
    __syncthreads();
    if (w != 0 || col >= s.dim) return;
#pragma unroll
    for (int e = 0; e < kCols; ++e) sum[e] = 0.0f;
    add_part(q.part + (2 * c + 1) * s.dim, s.dim, col, sum);
#pragma unroll
    for (int e = 0; e < kCols; ++e)
#pragma unroll
        for (int k = 0; k < kThreads / 64; ++k) sum[e] += quarter[k][lane * kCols + e];
    emit<DST>(grad, s, id, col, sum, scale, overwrite);
}

// ------------------------------------------------------------ host ---------
bool valid_type(int32_t dt) { return dt == ZERO_FP32 || dt == ZERO_FP16 || dt == ZERO_BF16; }
int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }
bool misaligned(const void* p, int32_t dt) { return (uintptr_t)p % (dt == ZERO_FP32 ? 4 : 2) != 0; }

int check_sizes(int64_t n_tokens, int64_t vocab, int64_t dim) {
    if (n_tokens < 0 || vocab < 1 || dim < 1) return ZERO_EINVAL;
    if (n_tokens > INT32_MAX || vocab > INT32_MAX - 1 || dim > INT32_MAX / 4) return ZERO_ERANGE;
    return ZERO_OK;
}
int check_slice(int64_t vocab, int64_t dim, int64_t begin, int64_t count) {
    if (begin < 0 || count < 0 || begin > vocab * dim || count > vocab * dim - begin) return ZERO_EINVAL;
    return ZERO_OK;
}

// Tokens of a chunk: enough chunks to fill the device, few enough that an id that
// most tokens have is added up in two short passes.
int64_t chunk_for(int64_t n, int64_t slabs) {
    int64_t c = kLeastChunk;
    while (c < kMostChunk && n * slabs > c * kChunkUnits) c *= 2;
    return c;
}
// A bound of the chunks of up to n tokens, so that a workspace for n serves fewer.
int64_t most_chunks(int64_t n, int64_t slabs) {
    const int64_t few = (n + kLeastChunk - 1) / kLeastChunk, full = kChunkUnits / slabs + 1;
    const int64_t many = (n + kMostChunk - 1) / kMostChunk;
    return many > full ? many : few < full ? few : full;
}
struct Layout {
    int64_t key[2], pos[2], counts, n_valid, part, bytes;
    int64_t chunk, chunks, slabs, blocks;
};
Layout layout_for(int64_t n, int64_t dim) {
    Layout l;
    l.slabs = (dim + kSlab - 1) / kSlab;
    l.chunk = chunk_for(n, l.slabs);
    l.chunks = (n + l.chunk - 1) / l.chunk;
    l.blocks = (n + kSortTile - 1) / kSortTile;
    int64_t at = 0;
    for (int k = 0; k < 2; ++k) {
        l.key[k] = at, at = up(at + 4 * n, 256);
        l.pos[k] = at, at = up(at + 4 * n, 256);
    }
    l.counts = at, at = up(at + 4 * kBins * l.blocks, 256);
    l.n_valid = at, at = up(at + 4, 256);
    l.part = at, at = up(at + 8 * most_chunks(n, l.slabs) * dim, 256);
    l.bytes = at;
    return l;
}

// go(first block, blocks) for pieces of a launch, in order.
template <typename F>
int in_pieces(int64_t blocks, F&& go) {
    for (int64_t b = 0; b < blocks; b += kMaxLaunchBlocks) {
        const int rc = go(b, blocks - b < kMaxLaunchBlocks ? blocks - b : kMaxLaunchBlocks);
        if (rc != ZERO_OK) return rc;
    }
    return ZERO_OK;
}

template <int DT>
struct Type {
    static constexpr int value = DT;
};
template <typename F>
int by_type(int32_t dt, F&& go) {
    return dt == ZERO_FP32 ? go(Type<ZERO_FP32>{}) : dt == ZERO_FP16 ? go(Type<ZERO_FP16>{}) : go(Type<ZERO_BF16>{});
}

}  // namespace

extern "C" {

int zero_embedding_lookup(void* out, int64_t out_ld, int32_t out_dtype, const void* ids, int32_t id_bytes,
                          int64_t n_tokens, const void* table, int32_t table_dtype, int64_t vocab, int64_t dim,
                          int64_t begin, int64_t count, float scale, hipStream_t stream) {
    if (const int rc = check_sizes(n_tokens, vocab, dim)) return rc;
    if (const int rc = check_slice(vocab, dim, begin, count)) return rc;
    if (!valid_type(out_dtype) || !valid_type(table_dtype) || (id_bytes != 4 && id_bytes != 8) ||
        out_ld < dim || !isfinite(scale))
        return ZERO_EINVAL;
    if (n_tokens == 0) return ZERO_OK;
    int64_t extent;
    if (__builtin_mul_overflow(out_ld, 4 * n_tokens, &extent)) return ZERO_ERANGE;
    if (!out || !ids || (count > 0 && !table) || (uintptr_t)ids % id_bytes || misaligned(out, out_dtype) ||
        misaligned(table, table_dtype))
        return ZERO_EINVAL;
    const Slice s = {vocab, dim, begin, count};
    const int64_t parts = (dim + kLookupCols - 1) / kLookupCols;
    return by_type(table_dtype, [&](auto src) {
        return by_type(out_dtype, [&](auto dst) {
            return in_pieces((n_tokens * parts + 3) / 4, [&](int64_t b, int64_t grid) {
                return launch(embedding_lookup_kernel<decltype(src)::value, decltype(dst)::value>, grid, 0, stream,
                              out, out_ld, ids, id_bytes == 8, n_tokens, (uint32_t)parts, table, s, scale, b);
            });
        });
    });
}

size_t zero_embedding_workspace_bytes(int64_t n_tokens, int64_t vocab, int64_t dim) {
    if (check_sizes(n_tokens, vocab, dim) != ZERO_OK) return 0;
    return (size_t)layout_for(n_tokens, dim).bytes;
}

int zero_embedding_grad(void* grad, int32_t grad_dtype, const void* ids, int32_t id_bytes, int64_t n_tokens,
                        const void* dy, int64_t dy_ld, int32_t dy_dtype, int64_t vocab, int64_t dim,
                        int64_t begin, int64_t count, int64_t padding_id, float scale, int32_t overwrite,
                        void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (const int rc = check_sizes(n_tokens, vocab, dim)) return rc;
    if (const int rc = check_slice(vocab, dim, begin, count)) return rc;
    if (!valid_type(grad_dtype) || !valid_type(dy_dtype) || (id_bytes != 4 && id_bytes != 8) || dy_ld < dim ||
        !isfinite(scale))
        return ZERO_EINVAL;
    if (count == 0 || (n_tokens == 0 && !overwrite)) return ZERO_OK;
    int64_t extent;
    if (__builtin_mul_overflow(dy_ld, 4 * n_tokens, &extent)) return ZERO_ERANGE;
    if (!grad || misaligned(grad, grad_dtype)) return ZERO_EINVAL;
    if (n_tokens > 0 && (!ids || !dy || (uintptr_t)ids % id_bytes || misaligned(dy, dy_dtype))) return ZERO_EINVAL;
    const Layout l = layout_for(n_tokens, dim);
    if (n_tokens > 0 && (!workspace || (uintptr_t)workspace % 256 || workspace_bytes < (size_t)l.bytes))
        return ZERO_EINVAL;
    char* ws = (char*)workspace;
    uint32_t* n_valid = n_tokens > 0 ? (uint32_t*)(ws + l.n_valid) : nullptr;
    const Slice s = {vocab, dim, begin, count};
    Keys keys = {ids, id_bytes == 8, n_tokens, padding_id < 0 ? -1 : padding_id, s};
    // passes of at most kDigit bits over the keys 0 .. vocab
    int bits = 1;
    while ((vocab >> bits) != 0) ++bits;
    const int passes = (bits + kDigit - 1) / kDigit, per = (bits + passes - 1) / passes;
    int at = 0;                                     // where the sorted tokens are
    int rc = ZERO_OK;
    if (n_tokens > 0 && n_tokens <= kSmallSort) {
        rc = launch_shape(embedding_sort_small_kernel, 1, kSortLanes, 0, stream, keys, passes, per,
                          (uint32_t*)(ws + l.key[0]), (uint32_t*)(ws + l.pos[0]), n_valid);
    } else if (n_tokens > 0) {
        uint32_t* counts = (uint32_t*)(ws + l.counts);
        for (int p = 0; p < passes && rc == ZERO_OK; ++p) {
            const Pairs in = {p == 0 ? nullptr : (const uint32_t*)(ws + l.key[at]),
                              p == 0 ? nullptr : (const uint32_t*)(ws + l.pos[at])};
            const int to = p == 0 ? 0 : at ^ 1;
            rc = launch_shape(embedding_count_kernel, l.blocks, kBigLanes, 0, stream, keys, in, p * per, per,
                              l.blocks, counts);
            const bool scan = l.blocks > kFewBlocks;
            if (rc == ZERO_OK && scan)
                rc = launch_shape(embedding_scan_kernel, 1, kSortLanes, 0, stream, counts, l.blocks << per);
            if (rc == ZERO_OK)
                rc = launch_shape(embedding_scatter_kernel, l.blocks, kBigLanes, 0, stream, keys, in, p * per, per,
                                  l.blocks, (const uint32_t*)counts, (int)scan, (uint32_t*)(ws + l.key[to]),
                                  (uint32_t*)(ws + l.pos[to]));
            at = to;
        }
        if (rc == ZERO_OK)
            rc = launch_shape(embedding_valid_kernel, 1, 64, 0, stream, (const uint32_t*)(ws + l.key[at]), n_tokens,
                              (uint32_t)vocab, n_valid);
    }
    if (rc != ZERO_OK) return rc;
    const Sorted q = {(const uint32_t*)(ws + l.key[at]), (const uint32_t*)(ws + l.pos[at]), n_valid, l.chunks,
                      (uint32_t)l.slabs, (float*)(ws + l.part), 0, 0};
    const int64_t size = grad_dtype == ZERO_FP32 ? 4 : 2;
    int rows = 64;                                   // of a wave that clears
    while (rows > 1 && rows * dim * size > kClearBytes) rows /= 2;
    const int64_t all_rows = (begin + count + dim - 1) / dim - begin / dim;
    const int64_t clear = overwrite ? ((all_rows + rows - 1) / rows + 3) / 4 : 0;
    const int64_t blocks = clear + (l.chunks * l.slabs + 3) / 4;
    rc = by_type(dy_dtype, [&](auto src) {
        return by_type(grad_dtype, [&](auto dst) {
            return in_pieces(blocks, [&](int64_t b, int64_t grid) {
                return launch(embedding_sum_kernel<decltype(src)::value, decltype(dst)::value>, grid, 0, stream, q,
                              dy, dy_ld, grad, s, scale, overwrite != 0, clear, rows, b);
            });
        });
    });
    if (rc != ZERO_OK || l.chunks < 2) return rc;
    return by_type(grad_dtype, [&](auto dst) {
        return in_pieces((l.chunks - 1) * l.slabs, [&](int64_t b, int64_t grid) {
            return launch(embedding_join_kernel<decltype(dst)::value>, grid, 0, stream, q, grad, s, scale,
                          overwrite != 0, b);
        });
    });
}

}  // extern "C"
