// Writing rows into the 4-bit K/V cache and reading them back.
//
// Both are one pass over the data, bound by HBM at large sizes and by the
// launch at a block's 32 rows: the store reads d * esize bytes per row and
// writes d/2 + d/16, the load the reverse. A thread handles 16 bytes of the
// unquantised row (8 bf16 or 4 f32 values), so 2 or 4 neighbouring lanes share
// a group and combine their maxima by shuffles, and every access of a warp is
// contiguous. The position is the fastest index after the row's pieces: the
// cache rows of one (sequence, head) are contiguous, and partial sectors (8 or
// 4 scale bytes per row) are filled by one warp.
#include "common.cuh"
#include "kv4.cuh"
#include "launch.h"

namespace fdl {

namespace {

constexpr int KV4_THREADS = 256;

struct Kv4RowsArgs {
    const void *k_src, *v_src;   // store: the fresh rows
    void *k_dst, *v_dst;         // load: the rows read back (null: not wanted)
    Kv4Ptrs c;
    long long seq_stride, row_stride, head_stride;   // of the rows, in elements
    int heads, L, start, n;
    uint32_t items;              // per sequence: heads * n * pieces of a row
    FastDiv by_n;
};

template <typename T> struct Piece { static constexpr int N = 16 / sizeof(T); };

__device__ __forceinline__ void unpack(const uint4& w, float (&v)[8]) {     // 8 bf16
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack(const uint4& w, float (&v)[4]) {     // 4 f32
    v[0] = __uint_as_float(w.x);
    v[1] = __uint_as_float(w.y);
    v[2] = __uint_as_float(w.z);
    v[3] = __uint_as_float(w.w);
}

// Quantise the N values of this lane, whose group of 16 lies in 16 / N
// neighbouring lanes (all of which call this); returns the codes, *scale the byte.
template <int N>
__device__ __forceinline__ uint32_t quantise(float (&v)[N], uint32_t* scale) {
    // the maximum of |x| as unsigned bits, which orders NaN above everything
    uint32_t mb = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) mb = max(mb, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
    for (int o = 1; o < KV4_GROUP / N; o <<= 1) mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, o));
    // max / 6 and x / scale as products with a reciprocal held in two floats
    // (fma(x, hi, x * lo), after Brisebarre and Muller): a quotient on the
    // border of two codes stays on it, where a single reciprocal's rounding
    // error moved 162 of the bf16 ties to the wrong side. A quotient next to
    // a border differs from it by more than its rounding.
    const float mx = __uint_as_float(mb);
    constexpr float sixth_hi = 1.f / 6.f;
    constexpr float sixth_lo = (float)(1.0 / 6.0 - (double)sixth_hi);
    float q = fmaf(mx, sixth_hi, mx * sixth_lo);
    if (mb >= 0x7f800000u) {                     // Inf saturates, NaN marks its group
        q = mx;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = fminf(fmaxf(v[i], -3.4e38f), 3.4e38f);
    }
    *scale = e4m3_byte(q);
    const float s = e4m3_f32(*scale);
    float hi = 0.f, lo = 0.f;
    if (s > 0.f) {
        hi = __frcp_rn(s);
        lo = fmaf(-s, hi, 1.f) * hi;
    }
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = i < N ? fmaf(v[i < N ? i : 0], hi, v[i < N ? i : 0] * lo) : 0.f;
    return e2m1x8(r);
}

// Where item e of sequence bb lies: its row's cache index, its offset among the
// unquantised rows (elements) and its piece of the row.
template <int D, int N>
struct Place {
    size_t row;
    long long at;
    uint32_t piece;
    __device__ __forceinline__ Place(const Kv4RowsArgs& a, int bb, uint32_t e) {
        constexpr uint32_t P = D / N;
        piece = e % P;
        const uint32_t hr = e / P, h = a.by_n.div(hr), i = hr - h * (uint32_t)a.n;
        row = ((size_t)bb * a.heads + h) * a.L + a.start + i;
        at = bb * a.seq_stride + i * a.row_stride + h * a.head_stride + piece * N;
    }
};

template <typename T, int D>
__global__ void __launch_bounds__(KV4_THREADS)
kv4_store_kernel(const Kv4RowsArgs a) {
    constexpr int N = Piece<T>::N, U = 2;
    constexpr int LANES = KV4_GROUP / N;         // lanes of a group
    pdl_wait();
    pdl_trigger();
    const bool is_v = blockIdx.y != 0;
    const int bb = blockIdx.z;
    const T* src = reinterpret_cast<const T*>(is_v ? a.v_src : a.k_src);
    uint8_t* all_codes = is_v ? a.c.v : a.c.k;
    uint8_t* all_scales = is_v ? a.c.v_scale : a.c.k_scale;
    // items is a multiple of LANES and of the pieces of a row: a group's lanes
    // are in range together, and the loop's bound below is uniform in a warp
    const uint32_t base = blockIdx.x * (KV4_THREADS * U) + (threadIdx.x & ~31u) * U +
                          (threadIdx.x & 31u);
    uint4 w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t e = base + u * 32;
        w[u] = make_uint4(0, 0, 0, 0);
        if (e < a.items) {
            const Place<D, N> p(a, bb, e);
            w[u] = __ldcs(reinterpret_cast<const uint4*>(src + p.at));
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t e = base + u * 32;
        float v[N];
        unpack(w[u], v);
        uint32_t sc;
        const uint32_t codes = quantise<N>(v, &sc);
        if (e >= a.items) continue;
        const Place<D, N> p(a, bb, e);
        uint8_t* c = all_codes + p.row * (D / 2) + p.piece * (N / 2);
        if (N == 8) *reinterpret_cast<uint32_t*>(c) = codes;
        else *reinterpret_cast<uint16_t*>(c) = (uint16_t)codes;
        if (p.piece % LANES == 0)
            all_scales[p.row * (D / KV4_GROUP) + p.piece / LANES] = (uint8_t)sc;
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(KV4_THREADS)
kv4_load_kernel(const Kv4RowsArgs a) {
    constexpr int N = Piece<T>::N, U = 4;
    constexpr int LANES = KV4_GROUP / N;
    pdl_wait();
    pdl_trigger();
    const bool is_v = blockIdx.y != 0;
    const int bb = blockIdx.z;
    T* dst = reinterpret_cast<T*>(is_v ? a.v_dst : a.k_dst);
    const uint8_t* all_codes = is_v ? a.c.v : a.c.k;
    const uint8_t* all_scales = is_v ? a.c.v_scale : a.c.k_scale;
    if (!dst) return;
    const uint32_t base = blockIdx.x * (KV4_THREADS * U) + (threadIdx.x & ~31u) * U +
                          (threadIdx.x & 31u);
    uint32_t w[U], sc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t e = base + u * 32;
        w[u] = sc[u] = 0;
        if (e < a.items) {
            const Place<D, N> p(a, bb, e);
            const uint8_t* c = all_codes + p.row * (D / 2) + p.piece * (N / 2);
            w[u] = N == 8 ? *reinterpret_cast<const uint32_t*>(c)
                          : *reinterpret_cast<const uint16_t*>(c);
            sc[u] = all_scales[p.row * (D / KV4_GROUP) + p.piece / LANES];
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t e = base + u * 32;
        if (e >= a.items) continue;
        const Place<D, N> p(a, bb, e);
        uint32_t h[N / 2];
        if constexpr (N == 8) e2m1x8_half2(w[u], h);
        else e2m1x4_half2((uint16_t)w[u], h);
        const float s = e4m3_f32(sc[u]);
        float v[N];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
            v[2 * i] = f.x * s;                  // at most 6 significant bits: exact
            v[2 * i + 1] = f.y * s;
        }
        uint4 o;
        if constexpr (N == 8) {
            uint32_t b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                b[i] = *reinterpret_cast<const uint32_t*>(&t);
            }
            o = make_uint4(b[0], b[1], b[2], b[3]);
        } else {
            o = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                           __float_as_uint(v[3]));
        }
        *reinterpret_cast<uint4*>(dst + p.at) = o;
    }
}

template <bool STORE>
cudaError_t launch_rows(const Kv4Rows& s, const void* k_src, const void* v_src, void* k_dst,
                        void* v_dst, const Kv4Ptrs& c, cudaStream_t st) {
    const int piece = s.bf16 ? 8 : 4, per_block = KV4_THREADS * (STORE ? 2 : 4);
    const uint32_t items = (uint32_t)s.heads * s.n * (s.head_dim / piece);
    Kv4RowsArgs a{k_src, v_src, k_dst, v_dst, c,
                  s.seq_stride, s.row_stride, s.head_stride,
                  s.heads, s.seq_len, s.start, s.n, items, FastDiv((uint32_t)s.n)};
    void (*kfn)(const Kv4RowsArgs);
    if constexpr (STORE)
        kfn = s.bf16 ? (s.head_dim == 128 ? kv4_store_kernel<bf16, 128> : kv4_store_kernel<bf16, 64>)
                     : (s.head_dim == 128 ? kv4_store_kernel<float, 128>
                                          : kv4_store_kernel<float, 64>);
    else
        kfn = s.bf16 ? (s.head_dim == 128 ? kv4_load_kernel<bf16, 128> : kv4_load_kernel<bf16, 64>)
                     : (s.head_dim == 128 ? kv4_load_kernel<float, 128>
                                          : kv4_load_kernel<float, 64>);
    const dim3 grid((items + per_block - 1) / per_block, 2, s.batch);
    return launch_pdl(kfn, grid, dim3(KV4_THREADS), 0, st, 0, a);
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
