// Writing rows into the 4-bit K/V cache and reading them back.
//
// Both are one pass over the data, bound by HBM at large sizes and by the
// launch at a block's 32 rows: the store reads d * esize bytes per row and
// writes d/2 + d/16, the load the reverse. A thread of the store has a group of
// 16 values, so a scale is found once; a thread of the load has 16 bytes of the
// row that it writes. A block lies within one sequence and covers whole heads or
// a piece of one, so a thread's addresses come from one multiplication and
// constant steps. Both are near their instruction limit, too: with half a group
// per thread (its scale found twice) the store issued 128 instructions for 8
// values, 83 % of the slots, and with a flat index divided for every access it
// took 23.8 us and the load 16.8 for 32 sequences of 4 x 1024 rows of 128 bf16
// (86 MB each way); now 13.7 and 14.6 us, 6.3 and 5.9 TB/s, 0.96 and 0.90 of the measured
// HBM rate. A block of 32 rows of 32 heads takes 1.7 us either way.
#include "common.cuh"
#include "kv4.cuh"
#include "launch.h"

namespace fdl {

namespace {

constexpr int KV4_THREADS = 256;
constexpr int LOAD_UNROLL = 4;                   // pieces per thread of the load

struct Kv4RowsArgs {
    const void *k_src, *v_src;   // store: the fresh rows
    void *k_dst, *v_dst;         // load: the rows read back (null: not wanted)
    Kv4Ptrs c;
    long long seq_stride, row_stride, head_stride;   // of the rows, in elements
    int heads, L, start, n;
    int head_blocks;             // blocks along the heads (grid.y is twice that: K, then V)
};

template <typename T> struct Piece { static constexpr int N = 16 / sizeof(T); };

// A group of 16 values as loaded: 2 (bf16) or 4 (f32) 16-byte words.
template <typename T> struct Group { uint4 w[sizeof(T)]; };

// Largest |x| of a group as float bits; NaN is above everything.
__device__ __forceinline__ uint32_t max_bits(const Group<bf16>& g) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        m = bf16x2_max_abs(bf16x2_max_abs(m, g.w[i].x), g.w[i].y);
        m = bf16x2_max_abs(bf16x2_max_abs(m, g.w[i].z), g.w[i].w);
    }
    return bf16x2_max_bits(m);
}
__device__ __forceinline__ uint32_t max_bits(const Group<float>& g) {
    uint32_t m = 0;
    const uint32_t a = 0x7fffffffu;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m = max(m, max(max(g.w[i].x & a, g.w[i].y & a), max(g.w[i].z & a, g.w[i].w & a)));
    return m;
}

__device__ __forceinline__ void unpack(const Group<bf16>& g, float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t u[4] = {g.w[i].x, g.w[i].y, g.w[i].z, g.w[i].w};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            v[8 * i + 2 * y] = __uint_as_float(u[y] << 16);
            v[8 * i + 2 * y + 1] = __uint_as_float(u[y] & 0xffff0000u);
        }
    }
}
__device__ __forceinline__ void unpack(const Group<float>& g, float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[4 * i] = __uint_as_float(g.w[i].x);
        v[4 * i + 1] = __uint_as_float(g.w[i].y);
        v[4 * i + 2] = __uint_as_float(g.w[i].z);
        v[4 * i + 3] = __uint_as_float(g.w[i].w);
    }
}

// Two products with hi + lo: fma(x, hi, fma(x, lo, 0)).
__device__ __forceinline__ void scale_pair(float& x, float& y, float hi, float lo) {
    asm("{\n\t.reg .b64 v, h, l, z;\n\t"
        "mov.b64 v, {%0, %1};\n\t"
        "mov.b64 h, {%2, %2};\n\t"
        "mov.b64 l, {%3, %3};\n\t"
        "mov.b64 z, {%4, %4};\n\t"
        "fma.rn.f32x2 l, v, l, z;\n\t"
        "fma.rn.f32x2 v, v, h, l;\n\t"
        "mov.b64 {%0, %1}, v;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(hi), "f"(lo), "f"(0.f));
}

// The codes of a group, and its scale byte.
template <typename T>
__device__ __forceinline__ uint2 quantise(const Group<T>& g, uint32_t* scale) {
    float v[16];
    unpack(g, v);
    const uint32_t mb = max_bits(g);
    // max / 6 and x / scale as products with a reciprocal held in two floats
    // (fma(x, hi, x * lo), after Brisebarre and Muller): a quotient on the
    // border of two codes stays on it, where a single reciprocal's rounding
    // error moved 162 of the bf16 ties to the wrong side (and for three of the
    // eight significands of a scale no single one keeps them all). A quotient
    // next to a border differs from it by more than its rounding.
    // The + 0 of the inner one makes every sum of zeros a +0, so that -0 has code 0, and
    // all of a group whose reciprocal is 0, where a product alone would keep its sign.
    // (Signs cleared in the codes instead: 32 sequences 15.4 us.)
    const float mx = __uint_as_float(mb);
    constexpr float sixth_hi = 1.f / 6.f;
    constexpr float sixth_lo = (float)(1.0 / 6.0 - (double)sixth_hi);
    float q = fmaf(mx, sixth_hi, mx * sixth_lo);
    if (mb >= 0x7f800000u) {                     // Inf saturates, NaN marks its group
        q = mx;
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = fminf(fmaxf(v[i], -3.4e38f), 3.4e38f);
    }
    *scale = e4m3_byte(q);
    const float s = e4m3_f32(*scale);
    float hi = 0.f, lo = 0.f;
    if (s > 0.f) {
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(hi) : "f"(s));
        lo = fmaf(-s, hi, 1.f) * hi;             // what hi lacks
    }
#pragma unroll
    for (int i = 0; i < 16; i += 2) scale_pair(v[i], v[i + 1], hi, lo);
    return make_uint2(e2m1x8(v), e2m1x8(v + 8));
}

// Where a thread works: blockDim = (pieces of a head at a time, heads at a time).
template <int D, int N>
struct Place {
    static constexpr int P = D / N;              // pieces of a row
    bool is_v, head_ok;
    int i, step, n;                              // first row, rows to the next piece, rows in all
    uint32_t piece;
    size_t row;                                  // cache row of the first
    long long at;                                // its piece's offset among the unquantised rows
    __device__ __forceinline__ Place(const Kv4RowsArgs& a, int unroll) {
        is_v = blockIdx.y >= (unsigned)a.head_blocks;
        const int h = (int)(blockIdx.y - (is_v ? a.head_blocks : 0)) * blockDim.y + threadIdx.y;
        const int bb = blockIdx.z;
        head_ok = h < a.heads;
        piece = threadIdx.x % P;
        step = blockDim.x / P;
        i = (int)blockIdx.x * step * unroll + threadIdx.x / P;
        n = a.n;
        row = ((size_t)bb * a.heads + h) * a.L + a.start + i;
        at = bb * a.seq_stride + (long long)h * a.head_stride + (long long)i * a.row_stride +
             piece * N;
    }
};

template <typename T, int D>
__global__ void __launch_bounds__(KV4_THREADS)
kv4_store_kernel(const Kv4RowsArgs a) {
    constexpr int U = 4 / sizeof(T);             // 64 bytes of rows per thread
    pdl_wait();
    pdl_trigger();
    const Place<D, KV4_GROUP> p(a, U);
    if (!p.head_ok) return;
    const T* src = reinterpret_cast<const T*>(p.is_v ? a.v_src : a.k_src) + p.at;
    uint2* codes = reinterpret_cast<uint2*>(p.is_v ? a.c.v : a.c.k) +
                   p.row * (D / KV4_GROUP) + p.piece;
    uint8_t* scales = (p.is_v ? a.c.v_scale : a.c.k_scale) + p.row * (D / KV4_GROUP) + p.piece;
    Group<T> g[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (p.i + u * p.step < p.n) {
            const uint4* at =
                reinterpret_cast<const uint4*>(src + (long long)u * p.step * a.row_stride);
#pragma unroll
            for (int i = 0; i < (int)sizeof(T); ++i) g[u].w[i] = __ldcs(at + i);
        }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (p.i + u * p.step >= p.n) break;
        uint32_t sc;
        codes[(size_t)(u * p.step) * (D / KV4_GROUP)] = quantise<T>(g[u], &sc);
        scales[(size_t)(u * p.step) * (D / KV4_GROUP)] = (uint8_t)sc;
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(KV4_THREADS)
kv4_load_kernel(const Kv4RowsArgs a) {
    constexpr int N = Piece<T>::N, U = LOAD_UNROLL;
    constexpr int LANES = KV4_GROUP / N;
    pdl_wait();
    pdl_trigger();
    const Place<D, N> p(a, U);
    T* dst = reinterpret_cast<T*>(p.is_v ? a.v_dst : a.k_dst);
    if (!dst || !p.head_ok) return;
    dst += p.at;
    const uint8_t* codes = (p.is_v ? a.c.v : a.c.k) + p.row * (D / 2) + p.piece * (N / 2);
    const uint8_t* scales = (p.is_v ? a.c.v_scale : a.c.k_scale) + p.row * (D / KV4_GROUP) +
                            p.piece / LANES;
    uint32_t w[U], sc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        w[u] = sc[u] = 0;
        if (p.i + u * p.step < p.n) {
            const uint8_t* c = codes + (size_t)(u * p.step) * (D / 2);
            w[u] = N == 8 ? *reinterpret_cast<const uint32_t*>(c)
                          : *reinterpret_cast<const uint16_t*>(c);
            sc[u] = scales[(size_t)(u * p.step) * (D / KV4_GROUP)];
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (p.i + u * p.step >= p.n) break;
        // code * scale is exact in f16, and then in T
        const uint32_t s2 = e4m3x2_half2(sc[u] * 0x0101u);
        uint32_t h[N / 2], o[4];
        if constexpr (N == 8) e2m1x8_half2(w[u], h);
        else e2m1x4_half2((uint16_t)w[u], h);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const uint32_t v = hmul2(h[i], s2);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
            if constexpr (N == 8) {
                const __nv_bfloat162 t = __floats2bfloat162_rn(f.x, f.y);
                o[i] = *reinterpret_cast<const uint32_t*>(&t);
            } else {
                o[2 * i] = __float_as_uint(f.x);
                o[2 * i + 1] = __float_as_uint(f.y);
            }
        }
        // streamed: 3.5 times the bytes read (19 MB to 67 MB: 14.6 us, without 16.6)
        __stcs(reinterpret_cast<uint4*>(dst + (long long)u * p.step * a.row_stride),
               make_uint4(o[0], o[1], o[2], o[3]));
    }
}

template <bool STORE>
cudaError_t launch_rows(const Kv4Rows& s, const void* k_src, const void* v_src, void* k_dst,
                        void* v_dst, const Kv4Ptrs& c, cudaStream_t st) {
    const int pieces = s.head_dim / (STORE ? KV4_GROUP : s.bf16 ? 8 : 4),
              unroll = !STORE ? LOAD_UNROLL : s.bf16 ? 2 : 1;
    // as many pieces of a head as there are, up to a block; the rest of the block
    // takes further heads
    const long long items = (long long)s.n * pieces;
    int x = KV4_THREADS;
    while (x > 32 && x / 2 * (long long)unroll >= items) x /= 2;
    const int y = KV4_THREADS / x, head_blocks = (s.heads + y - 1) / y;
    const long long rows = (long long)x / pieces * unroll;
    Kv4RowsArgs a{k_src, v_src, k_dst, v_dst, c,
                  s.seq_stride, s.row_stride, s.head_stride,
                  s.heads, s.seq_len, s.start, s.n, head_blocks};
    void (*kfn)(const Kv4RowsArgs);
    if constexpr (STORE)
        kfn = s.bf16 ? (s.head_dim == 128 ? kv4_store_kernel<bf16, 128>
                                          : kv4_store_kernel<bf16, 64>)
                     : (s.head_dim == 128 ? kv4_store_kernel<float, 128>
                                          : kv4_store_kernel<float, 64>);
    else
        kfn = s.bf16 ? (s.head_dim == 128 ? kv4_load_kernel<bf16, 128> : kv4_load_kernel<bf16, 64>)
                     : (s.head_dim == 128 ? kv4_load_kernel<float, 128>
                                          : kv4_load_kernel<float, 64>);
    const dim3 grid((unsigned)((s.n + rows - 1) / rows), 2 * head_blocks, s.batch);
    return launch_pdl(kfn, grid, dim3(x, y), 0, st, 0, a);
}

}  // namespace

cudaError_t launch_kv4_store(const Kv4Rows& s, const void* k_new, const void* v_new,
                             const Kv4Ptrs& c, cudaStream_t st) {
    return launch_rows<true>(s, k_new, v_new, nullptr, nullptr, c, st);
}

cudaError_t launch_kv4_load(const Kv4Rows& s, const Kv4Ptrs& c, void* k_out, void* v_out,
                            cudaStream_t st) {
    return launch_rows<false>(s, nullptr, nullptr, k_out, v_out, c, st);
}

}  // namespace fdl
