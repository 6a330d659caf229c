// Block attention over the 4-bit K/V cache.
//
// out = softmax(scale q K^T) V over the visible positions of each sequence,
// the same for all rows of its block: [0, sinks) and a window around the block,
// below the sequence's length. A kernel sees them as one run of indexes
// (Seen::pos maps an index to its position), so a window costs what it shows
// and no score is masked but those behind the end of a step.
//
// Everything between the cache and the output stays in registers. A warp takes
// steps of 32 visible positions and keeps a running maximum, sum and output of
// its own for the packed query rows (query i, head j of the kv head's group ->
// row i * G + j). The codes arrive by cp.async in the warp's own ring in shared
// memory (positions behind the end arrive as zeros: code 0 under scale 0), and
// each thread converts exactly the codes that its fragments of the matrix
// instructions need, so a cached value is converted once per 32 query rows and
// never written back to memory:
//   S = Q K^T   contraction over head_dim; the order of the dimensions is free
//               as long as Q has the same, so thread t of a quad owns dims
//               [D/4 t, D/4 (t+1)): one 16-byte load of a key's codes
//   O += P V    n = head_dim; thread group g owns dims [D/8 g, D/8 (g+1)), and
//               the codes of two neighbouring positions are interleaved nibble
//               by nibble before the conversion, so a converted byte is the
//               (position, position + 1) pair that the fragment wants
// The scores of a step go from the accumulators of the first product straight
// into the operand of the second; the position that column n of an 8-column
// tile stands for is chosen so that both products' loads are free of bank
// conflicts (row_of).
//
// Numbers: cached values are exact in f16 (kv4.cuh). Queries are brought to f16
// by a power of two per row that puts the row's largest value into
// [2^14, 2^15): exact down to 2^-29 of it. Probabilities are f16 with the
// running maximum at 2^7 to 2^15 (rescaled only when the maximum grows by more
// than 2^8), so that those below 2^-21 of the largest still have 11 bits. Sums,
// maxima and outputs are f32.
#include "common.cuh"
#include "kv4.cuh"
#include "launch.h"

namespace fdl {

namespace {

constexpr int A4_WARPS = 8, A4_THREADS = A4_WARPS * 32;
constexpr int A4_KS = 32;            // positions per step of a warp
constexpr int A4_STAGES = 3;
constexpr float A4_SHIFT = 7.f;      // log2 of a probability at the running maximum

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// c += A (16 x 16, rows) * B (16 x 8, columns), f16 with f32 sums.
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t* a, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool there) {
    const int n = there ? BYTES : 0;     // the rest is filled with zeros
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

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t r;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t a) {
    uint32_t r;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t a) {
    uint16_t r;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ void lds64(uint32_t a, uint32_t* r) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(a));
}
__device__ __forceinline__ void lds128(uint32_t a, uint32_t* r) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a));
}

struct Kv4AttnArgs {
    const bf16* q;
    const uint8_t *k, *ks, *v, *vs;
    bf16* out;
    float* lse;                  // optional
    float* part;                 // [unit][split][rows][D], with several splits
    float2* part_ml;             // [unit][split][rows]: running maximum, sum
    const int32_t* kv_len;       // optional
    int B, Hq, Hkv, G, L;
    int rows;                    // packed rows of a kv head: B * G
    int chunks, n_splits;
    int sinks, win_lo, win_hi;
    float scale_log2;
};

// The visible positions of one sequence: [0, first) and [lo, hi).
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

template <int D, int MT>
struct A4 {
    static constexpr int CB = D / 2, SB = D / KV4_GROUP;          // bytes of a row
    static constexpr int KK = D / 16;                             // k-steps of S
    static constexpr int NT = A4_KS / 8;                          // 8-column tiles of S
    static constexpr int ND = D / 8;                              // 8-column tiles of O
    static constexpr int ROWS = 16 * MT;
    static constexpr int OFF_K = 0, OFF_V = A4_KS * CB, OFF_KS = 2 * A4_KS * CB,
                         OFF_VS = OFF_KS + A4_KS * SB;
    static constexpr int STAGE = OFF_VS + A4_KS * SB;
    static constexpr int RING = A4_WARPS * A4_STAGES * STAGE;
    // after the steps the ring holds the warps' outputs, rows of D + 4 floats
    static constexpr int PROW = D + 4;
    static constexpr int PART = A4_WARPS * ROWS * PROW * 4;
    static constexpr int OFF_Q = RING > PART ? RING : PART;       // Q fragments
    static constexpr int OFF_RS = OFF_Q + MT * KK * 512;          // row scales
    static constexpr int OFF_ML = OFF_RS + ROWS * 4;              // warps' (max, sum)
    static constexpr int TOTAL = OFF_ML + A4_WARPS * ROWS * 8;
    static_assert(TOTAL <= 227 * 1024, "shared memory");
};

// Position (of the 8 of a tile) that column 2t + e of an S tile stands for: the
// second product's loads take four neighbouring positions per e, the first's
// take, per 8 lanes, two of different parity.
__device__ __forceinline__ int row_of(int t, int e) { return 4 * e + (t ^ e); }

// float4 slot of columns [4c, 4c + 4) in a partial row, so that the lanes of a
// quad, D/4 columns apart, and neighbouring rows write to different banks.
__device__ __forceinline__ int slot(int c) {
    return c ^ ((c >> 3) << 1);
}

template <int D, int MT>
__global__ void __launch_bounds__(A4_THREADS, 1)
kv4_attn_kernel(const Kv4AttnArgs a) {
    using S = A4<D, MT>;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sb = (uint32_t)__cvta_generic_to_shared(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    // block -> (sequence, kv head, row chunk, split)
    int u = blockIdx.x;
    const int split = u % a.n_splits;
    const int unit = u / a.n_splits;
    u = unit;
    const int chunk = u % a.chunks;
    u /= a.chunks;
    const int h = u % a.Hkv, bb = u / a.Hkv;
    const int row0 = chunk * S::ROWS;

    pdl_wait();
    pdl_trigger();

    const Seen seen(a, bb);
    // this split's run of indexes, whole steps but for the last
    const int steps_all = (seen.count + A4_KS - 1) / A4_KS;
    const int sps = (steps_all + a.n_splits - 1) / a.n_splits;
    const int i0 = min(split * sps, steps_all) * A4_KS;
    const int i1 = min(seen.count, i0 + sps * A4_KS);
    const int n_steps = i1 > i0 ? (i1 - i0 + A4_KS - 1) / A4_KS : 0;
    const int mine = n_steps > warp ? (n_steps - warp + A4_WARPS - 1) / A4_WARPS : 0;

    const size_t head = ((size_t)bb * a.Hkv + h) * a.L;
    const uint8_t* kc = a.k + head * S::CB;
    const uint8_t* vc = a.v + head * S::CB;
    const uint8_t* ks = a.ks + head * S::SB;
    const uint8_t* vs = a.vs + head * S::SB;
    const uint32_t ring = sb + warp * (A4_STAGES * S::STAGE);

    auto request = [&](int n) {              // the n-th step of this warp
        if (n < mine) {
            const uint32_t st = ring + (n % A4_STAGES) * S::STAGE;
            const int base = i0 + (warp + n * A4_WARPS) * A4_KS;
            constexpr int CH = S::CB / 16;   // 16-byte pieces of a row
#pragma unroll
            for (int x = 0; x < A4_KS * CH / 32; ++x) {
                const int e = lane + 32 * x, row = e / CH, ch = e % CH;
                const bool there = base + row < i1;
                const size_t off = (size_t)(there ? seen.pos(base + row) : 0) * S::CB + ch * 16;
                // the halves of a row swapped on every second pair of rows
                const uint32_t to = row * S::CB + ((CH == 4 ? ch ^ (row & 2) : ch) << 4);
                cp_async<16>(st + S::OFF_K + to, kc + off, there);
                cp_async<16>(st + S::OFF_V + to, vc + off, there);
            }
            const bool there = base + lane < i1;
            const size_t off = (size_t)(there ? seen.pos(base + lane) : 0) * S::SB;
            cp_async<S::SB>(st + S::OFF_KS + lane * S::SB, ks + off, there);
            cp_async<S::SB>(st + S::OFF_VS + lane * S::SB, vs + off, there);
        }
        cp_commit();                         // empty groups keep the count
    };
#pragma unroll
    for (int n = 0; n < A4_STAGES - 1; ++n) request(n);

    // Q fragments: row r of the chunk by warp r % 8; a lane has D / 32 of its
    // dims. Fragment word (mt, kk, lane (g, t), w): row mt*16 + g + 8*(w & 1),
    // dims D/4 t + 4 kk + 2 (w >> 1), +1.
    for (int r = warp; r < S::ROWS; r += A4_WARPS) {
        const int pr = row0 + r;
        float x[D / 32];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) x[i] = 0.f;
        if (pr < a.rows) {
            const int i = pr / a.G, j = pr - i * a.G;
            const bf16* src = a.q + (((size_t)bb * a.B + i) * a.Hq + h * a.G + j) * D +
                              lane * (D / 32);
            uint32_t w[D / 64];
            if constexpr (D == 128) {
                const uint2 v = *reinterpret_cast<const uint2*>(src);
                w[0] = v.x;
                w[1] = v.y;
            } else {
                w[0] = *reinterpret_cast<const uint32_t*>(src);
            }
#pragma unroll
            for (int k = 0; k < D / 64; ++k) {
                x[2 * k] = __uint_as_float(w[k] << 16);
                x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
            }
        }
        uint32_t mb = 0;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) mb = max(mb, __float_as_uint(x[i]) & 0x7fffffffu);
        mb = __reduce_max_sync(0xffffffffu, mb);
        // 2^(14 - exponent); 1 for a row of zeros, Inf or NaN
        const int ex = (int)(mb >> 23);
        float f = 1.f, inv = 1.f;
        if (mb != 0 && ex < 255) {
            const int p = min(14 + 127 - ex, 126);
            f = __uint_as_float((uint32_t)(127 + p) << 23);
            inv = __uint_as_float((uint32_t)(127 - p) << 23);
        }
        // at least the smallest normal number: a score of -inf times it stays so
        if (lane == 0)
            reinterpret_cast<float*>(smem + S::OFF_RS)[r] = fmaxf(a.scale_log2 * inv, 1.2e-38f);
#pragma unroll
        for (int k = 0; k < D / 64; ++k) {
            const int d = lane * (D / 32) + 2 * k;                // this pair's first dim
            const int qt = d / (D / 4), in = d % (D / 4);
            const int kk = in >> 2, w = ((r >> 3) & 1) | ((in >> 1) & 1) << 1;
            const int at = (((r >> 4) * S::KK + kk) * 32 + (r & 7) * 4 + qt) * 4 + w;
            reinterpret_cast<uint32_t*>(smem + S::OFF_Q)[at] =
                pack_half2(x[2 * k] * f, x[2 * k + 1] * f);
        }
    }
    __syncthreads();

    float rs[MT][2], m[MT][2], l[MT][2], o[MT][S::ND][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            rs[mt][x] = reinterpret_cast<const float*>(smem + S::OFF_RS)[mt * 16 + g + 8 * x];
            m[mt][x] = -INFINITY;
            l[mt][x] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < S::ND; ++j)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[mt][j][x] = 0.f;
    }

    for (int n = 0; n < mine; ++n) {
        cp_wait<A4_STAGES - 2>();
        __syncwarp();                        // the step is there, the last one's stage free
        request(n + A4_STAGES - 1);
        const uint32_t st = ring + (n % A4_STAGES) * S::STAGE;
        const int base = i0 + (warp + n * A4_WARPS) * A4_KS;

        // ---- S = Q K^T
        float s[MT][S::NT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < S::NT; ++nt)
#pragma unroll
                for (int x = 0; x < 4; ++x) s[mt][nt][x] = 0.f;
        {
            constexpr int W = D / 32;        // words of codes per thread and key
            uint32_t kw[S::NT][W], sc[S::NT];
            const int kr = row_of(g >> 1, g & 1);
#pragma unroll
            for (int nt = 0; nt < S::NT; ++nt) {
                const int row = 8 * nt + kr;
                const uint32_t ka = st + S::OFF_K + row * S::CB;
                if constexpr (D == 128) {
                    lds128(ka + ((t ^ (row & 2)) << 4), kw[nt]);
                    sc[nt] = lds_u16(st + S::OFF_KS + row * S::SB + 2 * t);
                } else {
                    lds64(ka + 8 * t, kw[nt]);
                    sc[nt] = lds_u8(st + S::OFF_KS + row * S::SB + t) * 0x0101u;
                }
                sc[nt] = e4m3x2_half2(sc[nt]);
            }
#pragma unroll
            for (int w = 0; w < W; ++w) {
                uint32_t qf[MT][2][4];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        lds128(sb + S::OFF_Q + ((mt * S::KK + 2 * w + x) * 32 + lane) * 16,
                               qf[mt][x]);
#pragma unroll
                for (int nt = 0; nt < S::NT; ++nt) {
                    uint32_t b[4];
                    e2m1x8_half2(kw[nt][w], b);
                    const uint32_t s2 = __byte_perm(sc[nt], 0, w < 2 ? 0x1010 : 0x3232);
#pragma unroll
                    for (int x = 0; x < 4; ++x) b[x] = hmul2(b[x], s2);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        mma16816(s[mt][nt], qf[mt][0], b[0], b[1]);
                        mma16816(s[mt][nt], qf[mt][1], b[2], b[3]);
                    }
                }
            }
        }

        // ---- softmax of the step; columns 2t + e of tile nt
        if (base + A4_KS > i1) {
#pragma unroll
            for (int nt = 0; nt < S::NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (base + 8 * nt + row_of(t, e) >= i1) {
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
                            s[mt][nt][e] = s[mt][nt][2 + e] = -INFINITY;
                    }
        }
        float mx[MT][2];
        bool grow = false;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float v = s[mt][0][2 * x];
#pragma unroll
                for (int nt = 0; nt < S::NT; ++nt)
                    v = fmaxf(v, fmaxf(s[mt][nt][2 * x], s[mt][nt][2 * x + 1]));
                mx[mt][x] = v * rs[mt][x];   // rs >= 0 commutes with the maximum
                grow |= mx[mt][x] > m[mt][x] + 8.f;
            }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float v = mx[mt][x];
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
                    const float mn = fmaxf(m[mt][x], v);
                    // nothing seen so far: l and o are zero and stay so
                    const float alpha = mn == -INFINITY ? 1.f : ex2(m[mt][x] - mn);
                    m[mt][x] = mn;
                    l[mt][x] *= alpha;
#pragma unroll
                    for (int j = 0; j < S::ND; ++j) {
                        o[mt][j][2 * x] *= alpha;
                        o[mt][j][2 * x + 1] *= alpha;
                    }
                }
        }
        uint32_t p[MT][S::NT][2];            // rows g and g + 8: the operand's pairs
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float nm = m[mt][x] == -INFINITY ? 0.f : A4_SHIFT - m[mt][x];
#pragma unroll
                for (int nt = 0; nt < S::NT; ++nt) {
                    const float p0 = ex2(fmaf(s[mt][nt][2 * x], rs[mt][x], nm));
                    const float p1 = ex2(fmaf(s[mt][nt][2 * x + 1], rs[mt][x], nm));
                    l[mt][x] += p0 + p1;
                    p[mt][nt][x] = pack_half2(p0, p1);
                }
            }

        // ---- O += P V, 16 positions (two S tiles) at a time
#pragma unroll
        for (int k = 0; k < S::NT / 2; ++k) {
            constexpr int W = D / 64;        // words of codes per thread and position
            uint32_t vw[2][2][W], s2[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                uint32_t sc[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = 8 * (2 * k + x) + row_of(t, e);
                    const uint32_t va = st + S::OFF_V + row * S::CB;
                    if constexpr (D == 128) {
                        lds64(va + ((((g >> 1) ^ (row & 2)) << 4) | ((g & 1) << 3)), vw[x][e]);
                        sc[e] = lds_u8(st + S::OFF_VS + row * S::SB + g);
                    } else {
                        vw[x][e][0] = lds32(va + 4 * g);
                        sc[e] = lds_u8(st + S::OFF_VS + row * S::SB + (g >> 1));
                    }
                }
                s2[x] = e4m3x2_half2(sc[0] | sc[1] << 8);
            }
#pragma unroll
            for (int w = 0; w < W; ++w) {
                // byte i: (position e = 0, position e = 1) of dim 2i (ev), 2i + 1 (od)
                uint32_t ev[2][4], od[2][4];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t c0 = vw[x][0][w], c1 = vw[x][1][w];
                    e2m1x8_half2((c0 & 0x0f0f0f0fu) | ((c1 << 4) & 0xf0f0f0f0u), ev[x]);
                    e2m1x8_half2(((c0 >> 4) & 0x0f0f0f0fu) | (c1 & 0xf0f0f0f0u), od[x]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        ev[x][i] = hmul2(ev[x][i], s2[x]);
                        od[x][i] = hmul2(od[x][i], s2[x]);
                    }
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const uint32_t pa[4] = {p[mt][2 * k][0], p[mt][2 * k][1],
                                            p[mt][2 * k + 1][0], p[mt][2 * k + 1][1]};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        mma16816(o[mt][8 * w + 2 * i], pa, ev[0][i], ev[1][i]);
                        mma16816(o[mt][8 * w + 2 * i + 1], pa, od[0][i], od[1][i]);
                    }
                }
            }
        }
    }
    cp_wait<0>();

    // ---- the warps' outputs joined in shared memory
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            l[mt][x] += __shfl_xor_sync(0xffffffffu, l[mt][x], 1);
            l[mt][x] += __shfl_xor_sync(0xffffffffu, l[mt][x], 2);
        }
    __syncthreads();                         // every warp has left its ring
    const int live = min(A4_WARPS, n_steps); // warps that took a step
    const int own = min(S::ROWS, a.rows - row0);
    float2* ml = reinterpret_cast<float2*>(smem + S::OFF_ML);
    if (warp < live) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int r = mt * 16 + g + 8 * x;
                if (r >= own) continue;
                float4* row = reinterpret_cast<float4*>(
                    reinterpret_cast<float*>(smem) + (size_t)(warp * S::ROWS + r) * S::PROW);
                // columns D/8 (2t + e) + j
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int j = 0; j < S::ND; j += 4)
                        row[slot((S::ND * (2 * t + e) + j) / 4)] =
                            make_float4(o[mt][j][2 * x + e], o[mt][j + 1][2 * x + e],
                                        o[mt][j + 2][2 * x + e], o[mt][j + 3][2 * x + e]);
                if (t == 0) ml[warp * S::ROWS + r] = make_float2(m[mt][x], l[mt][x]);
            }
    }
    __syncthreads();
    for (int it = threadIdx.x; it < own * (D / 4); it += A4_THREADS) {
        const int r = it / (D / 4), c = it % (D / 4);
        float M = -INFINITY;
        for (int w = 0; w < live; ++w) M = fmaxf(M, ml[w * S::ROWS + r].x);
        const float Ms = M == -INFINITY ? 0.f : M;
        float sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < live; ++w) {
            const float2 p = ml[w * S::ROWS + r];
            const float f = ex2(p.x - Ms);
            const float4 v = reinterpret_cast<const float4*>(
                reinterpret_cast<const float*>(smem) +
                (size_t)(w * S::ROWS + r) * S::PROW)[slot(c)];
            sum += p.y * f;
            acc.x += v.x * f;
            acc.y += v.y * f;
            acc.z += v.z * f;
            acc.w += v.w * f;
        }
        const int pr = row0 + r, i = pr / a.G, j = pr - i * a.G, qh = h * a.G + j;
        if (a.n_splits == 1) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;      // nothing visible: 0
            __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
            __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
            *reinterpret_cast<uint2*>(a.out + (((size_t)bb * a.B + i) * a.Hq + qh) * D + 4 * c) =
                make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
            if (a.lse && c == 0)
                a.lse[((size_t)bb * a.Hq + qh) * a.B + i] =
                    (Ms - A4_SHIFT + log2f(sum)) * 0.69314718055994530942f;
        } else {
            const size_t at = ((size_t)unit * a.n_splits + split) * S::ROWS + r;
            *reinterpret_cast<float4*>(a.part + at * D + 4 * c) = acc;
            if (c == 0) a.part_ml[at] = make_float2(M, sum);
        }
    }
}

// The splits' partial outputs joined: one warp per row.
template <int D, int ROWS>
__global__ void __launch_bounds__(256) kv4_join_kernel(const Kv4AttnArgs a, int units) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (item >= (long long)units * ROWS) return;
    const int unit = (int)(item / ROWS), r = (int)(item % ROWS);
    const int chunk = unit % a.chunks, h = unit / a.chunks % a.Hkv, bb = unit / a.chunks / a.Hkv;
    const int pr = chunk * ROWS + r;
    if (pr >= a.rows) return;
    const size_t at = (size_t)unit * a.n_splits * ROWS + r;
    float M = -INFINITY;
    for (int s = lane; s < a.n_splits; s += 32) M = fmaxf(M, a.part_ml[at + (size_t)s * ROWS].x);
    M = warp_max(M);
    const float Ms = M == -INFINITY ? 0.f : M;
    constexpr int E = D / 32;                // columns per lane
    float acc[E], sum = 0.f;
#pragma unroll
    for (int x = 0; x < E; ++x) acc[x] = 0.f;
#pragma unroll 4
    for (int s = 0; s < a.n_splits; ++s) {
        const float2 p = a.part_ml[at + (size_t)s * ROWS];
        const float f = ex2(p.x - Ms);
        const float* src = a.part + (at + (size_t)s * ROWS) * D + lane * E;
        sum += p.y * f;
        if constexpr (E == 4) {
            const float4 v = *reinterpret_cast<const float4*>(src);
            acc[0] += v.x * f;
            acc[1] += v.y * f;
            acc[2] += v.z * f;
            acc[3] += v.w * f;
        } else {
            const float2 v = *reinterpret_cast<const float2*>(src);
            acc[0] += v.x * f;
            acc[1] += v.y * f;
        }
    }
    const int i = pr / a.G, qh = h * a.G + pr - i * a.G;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    bf16* dst = a.out + (((size_t)bb * a.B + i) * a.Hq + qh) * D + lane * E;
#pragma unroll
    for (int x = 0; x < E; x += 2) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(acc[x] * inv, acc[x + 1] * inv);
        *reinterpret_cast<__nv_bfloat162*>(dst + x) = v;
    }
    if (a.lse && lane == 0)
        a.lse[((size_t)bb * a.Hq + qh) * a.B + i] =
            (Ms - A4_SHIFT + log2f(sum)) * 0.69314718055994530942f;
}

struct A4Plan {
    int mt, chunks, n_splits;
    long long units;
};

// The most positions that a sequence may see.
int most_seen(const Kv4Attn& s) {
    if (s.sinks >= s.win_lo) return s.sinks > s.win_hi ? s.sinks : s.win_hi;
    return s.sinks + s.win_hi - s.win_lo;
}

A4Plan a4_plan(const Kv4Attn& s, int sm_count) {
    A4Plan p;
    const int rows = s.block_len * (s.n_q_heads / s.n_kv_heads);
    p.mt = rows <= 16 ? 1 : 2;
    p.chunks = (rows + 16 * p.mt - 1) / (16 * p.mt);
    p.units = (long long)s.batch * s.n_kv_heads * p.chunks;
    const long long steps = (most_seen(s) + A4_KS - 1) / A4_KS;
    long long n = p.units < sm_count ? sm_count / p.units : 1;
    const long long most = (steps + A4_WARPS - 1) / A4_WARPS;   // a step for each warp
    p.n_splits = (int)(n > most ? most : n);
    if (p.n_splits < 1) p.n_splits = 1;
    return p;
}

template <int D, int MT>
cudaError_t run_a4(const Kv4AttnArgs& a, long long units, cudaStream_t st) {
    using S = A4<D, MT>;
    auto kfn = kv4_attn_kernel<D, MT>;
    cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         S::TOTAL);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kfn, dim3((unsigned)(units * a.n_splits)), dim3(A4_THREADS), S::TOTAL, st, 0, a);
    if (e != cudaSuccess || a.n_splits == 1) return e;
    const long long items = units * S::ROWS;
    return launch_pdl(kv4_join_kernel<D, S::ROWS>, dim3((unsigned)((items + 7) / 8)), dim3(256), 0,
                      st, 0, a, (int)units);
}

}  // namespace

size_t kv4_attention_workspace_bytes(const Kv4Attn& s, int sm_count) {
    const A4Plan p = a4_plan(s, sm_count);
    if (p.n_splits == 1) return 16;
    return (size_t)p.units * p.n_splits * 16 * p.mt * (s.head_dim * 4 + 8);
}

cudaError_t launch_kv4_attention(const Kv4Attn& s, const void* q, const Kv4Ptrs& c, void* out,
                                 float* lse, void* ws, int sm_count, cudaStream_t st) {
    const A4Plan p = a4_plan(s, sm_count);
    Kv4AttnArgs a{};
    a.q = (const bf16*)q;
    a.k = c.k;
    a.ks = c.k_scale;
    a.v = c.v;
    a.vs = c.v_scale;
    a.out = (bf16*)out;
    a.lse = lse;
    a.kv_len = s.kv_len;
    a.B = s.block_len;
    a.Hq = s.n_q_heads;
    a.Hkv = s.n_kv_heads;
    a.G = s.n_q_heads / s.n_kv_heads;
    a.L = s.seq_len;
    a.rows = a.B * a.G;
    a.chunks = p.chunks;
    a.n_splits = p.n_splits;
    a.sinks = s.sinks;
    a.win_lo = s.win_lo;
    a.win_hi = s.win_hi;
    a.scale_log2 = s.scale * 1.4426950408889634f;
    a.part = (float*)ws;
    a.part_ml = (float2*)((float*)ws + (size_t)p.units * p.n_splits * 16 * p.mt * s.head_dim);
    if (s.head_dim == 128)
        return p.mt == 1 ? run_a4<128, 1>(a, p.units, st) : run_a4<128, 2>(a, p.units, st);
    return p.mt == 1 ? run_a4<64, 1>(a, p.units, st) : run_a4<64, 2>(a, p.units, st);
}

}  // namespace fdl
