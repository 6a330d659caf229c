// What the kernels of the attention over the 4-bit K/V cache share.
#pragma once
#include "common.cuh"
#include "kv4.cuh"
#include "launch.h"

#include <atomic>

namespace fdl {

constexpr float KV4_SHIFT = 7.f;     // log2 of a probability at the running maximum

struct Kv4AttnArgs {
    const bf16* q;
    const uint8_t *k, *ks, *v, *vs;
    bf16* out;
    float* lse;                  // optional
    float* part;                 // [unit][part][chunk_rows][D], with several parts
    float4* part_ml;             // [unit][part][chunk_rows]: running maximum, sum, score scale
    const int32_t* kv_len;       // optional
    int B, Hq, Hkv, G, L;
    FastDiv by_g;
    int rows;                    // packed rows of a kv head, B * G: row i * G + j is query i
                                 // of head j of the kv head's group
    int chunks, chunk_rows;      // ... in chunks of at most so many
    int n_splits;                // splits of a unit (sequence, kv head, chunk), whole clusters
    int cluster;                 // splits that join on chip
    int parts;                   // n_splits / cluster: partial results left in the workspace
    int sinks, win_lo, win_hi;
    float scale_log2;
    int polled;                  // the context's wait limit is a shortened one
    int* err;
};

// The visible positions of one sequence, [0, first) and [lo, hi), as one run of
// indexes.
struct Seen {
    int first, gap, count;       // index i -> position i < first ? i : i + gap
    __device__ __forceinline__ Seen(const Kv4AttnArgs& a, int bb) {
        const int len = a.kv_len ? max(0, min(a.L, __ldg(a.kv_len + bb))) : a.L;
        const int hi = min(a.win_hi, len), lo = min(a.win_lo, hi), s = min(a.sinks, len);
        if (s < lo) {
            first = s;
            gap = lo - s;
            count = s + hi - lo;
        } else {                 // one run
            first = count = max(s, hi);
            gap = 0;
        }
    }
    __device__ __forceinline__ int pos(int i) const { return i < first ? i : i + gap; }
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// 16 bytes (or 4, 8) to shared memory, or as many zeros.
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool there) {
    const int n = there ? BYTES : 0;
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src),
                     "n"(BYTES), "r"(n)
                     : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Packed row pr of kv head h: its query, and the query head.
struct RowAt {
    int i, head;
    __device__ __forceinline__ RowAt(const Kv4AttnArgs& a, int h, int pr) {
        i = (int)a.by_g.div((uint32_t)pr);
        head = h * a.G + pr - i * a.G;
    }
    // element offset of the row in q and out, and the place of its log-sum-exp
    __device__ __forceinline__ size_t at(const Kv4AttnArgs& a, int bb, int D) const {
        return (((size_t)bb * a.B + i) * a.Hq + head) * D;
    }
    __device__ __forceinline__ size_t lse(const Kv4AttnArgs& a, int bb) const {
        return ((size_t)bb * a.Hq + head) * a.B + i;
    }
};

// The power of two that puts a row's largest magnitude (as float bits) into
// [2^14, 2^15), and its inverse; 1 for a row of zeros, Inf or NaN.
__device__ __forceinline__ void kv4_row_scale(uint32_t max_bits, float* f, float* inv) {
    const int ex = (int)(max_bits >> 23);
    *f = *inv = 1.f;
    if (max_bits != 0 && ex < 255) {
        const int p = min(14 + 127 - ex, 126);
        *f = __uint_as_float((uint32_t)(127 + p) << 23);
        *inv = __uint_as_float((uint32_t)(127 - p) << 23);
    }
}

// What a row's scores are multiplied with (rs below): at least the smallest normal
// number, so that a score of -inf stays one, and finite, so that a difference of 0
// stays one.
__device__ __forceinline__ float kv4_score_scale(float scale_log2, float inv) {
    return fminf(fmaxf(scale_log2 * inv, 1.2e-38f), 3.4028234663852886e38f);
}

// Maxima are kept in the scores' own units, and every exponent is a difference of two
// scores times rs: with a product m * rs that is rounded before the subtraction, the
// maximum's own exponent would be off by half an ulp of m * rs, which leaves f16's
// range where |m * rs| passes 2^27. Nothing seen (m = -inf) gives 2^-inf = 0.
__device__ __forceinline__ float kv4_base(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ float kv4_weight(float m, float base, float rs) {
    return ex2((m - base) * rs);
}
// log2 of two probabilities, (s - base) * rs + shift.
__device__ __forceinline__ float2 kv4_exponents(float s0, float s1, float base, float rs) {
    float2 r;
    asm("{\n\t.reg .b64 s, b, f, k;\n\t"
        "mov.b64 s, {%2, %3};\n\t"
        "mov.b64 b, {%4, %4};\n\t"
        "mov.b64 f, {%5, %5};\n\t"
        "mov.b64 k, {%6, %6};\n\t"
        "add.rn.f32x2 s, s, b;\n\t"
        "fma.rn.f32x2 s, s, f, k;\n\t"
        "mov.b64 {%0, %1}, s;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(s0), "f"(s1), "f"(-base), "f"(rs), "f"(KV4_SHIFT));
    return r;
}

// The log-sum-exp of a row from its maximum and sum.
__device__ __forceinline__ float kv4_lse(float m, float rs, float sum) {
    return fmaf(kv4_base(m), rs, log2f(sum) - KV4_SHIFT) * 0.69314718055994530942f;
}

// Few query rows per kv head (registers, mma.sync) and many (tcgen05).
cudaError_t launch_kv4_attn_few(const Kv4AttnArgs& a, const Kv4Plan& p, int head_dim,
                                cudaStream_t st);
cudaError_t launch_kv4_attn_many(const Kv4AttnArgs& a, const Kv4Plan& p, int head_dim,
                                 cudaStream_t st);

// The kernel's shared memory limit, set once per device.
template <typename K>
cudaError_t kv4_allow_smem(K kernel, size_t bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Clusters of c blocks (2 to 8) that the GPU holds at once: a cluster must fit in
// one GPC. Queried once, outside any stream capture (fdl_create); 0 while unknown.
int kv4_clusters(const void* kernel, int threads, size_t smem, int c, std::atomic<int>* known);
int kv4_few_clusters(int head_dim, int mt, int c);
int kv4_many_clusters(int head_dim, int mt, int c);

}  // namespace fdl
