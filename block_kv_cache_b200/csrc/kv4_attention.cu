// Block attention over the 4-bit K/V cache.
//
// out = softmax(scale q K^T) V over the visible positions of each sequence,
// the same for all rows of its block: [0, sinks) and a window around the block,
// below the sequence's length. A kernel sees them as one run of indexes
// (Seen::pos maps an index to its position), so a window costs what it shows
// and no score is masked but those behind the end of a step.
//
// Few query rows per kv head (a token's, a short block's): what it costs is reading
// and converting the cache, (16 + 2) / 16 bytes per 16 values of K and V, so all of
// it stays in registers between the two. A warp takes steps of 32 visible positions
// (16 with more than 16 rows) and keeps a running maximum, sum and output of its own
// for the packed query rows (query i, head j of the kv head's group -> row i * G + j).
// The codes arrive by cp.async in the warp's own ring in shared memory (positions
// behind the end arrive as zeros: code 0 under scale 0), and each thread converts
// exactly the codes that its fragments of the matrix instructions need, so a cached
// value is converted once per 32 query rows and never written back to memory. That
// is what mma.sync gives here and tcgen05 does not: its operands have to be stored
// to shared memory as f16, four times the bytes of the codes, and one of its tiles
// has 128 rows, of which 4 to 32 would be used (measured with positions as the rows
// instead: a token over 131072 positions 85 us, a 32 x 7 block over 768 10.9 us).
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
// The warps of a block join in shared memory, and the blocks of a cluster (the splits
// of one unit) by st.async into the block that finishes a row, which counts the bytes
// on a barrier. With more than 8 splits the clusters leave partial results in the
// workspace and a second kernel joins them.
//
// What bounds it (heads of 128; 6.55 TB/s measured copy): one token of 28 heads over
// 131072 positions of 4, 75.5 MB: 25.7 us with the join. 18 of them in the steps (4.2
// TB/s), where neither the issue slots (49 % over the whole kernel) nor the tensor pipe
// (32 %) are full: dependent work of four warps a scheduler, and 128 registers (20 bytes
// spilled) allow no fifth. Half of the 64 that hold outputs are rows 8 to 15, which the
// 7 heads of a group do not fill; the queries as the 8 columns would free them. 2.3
// before the first step, 2.4 for the join. A block of 32 rows over 768 positions: 7.8
// us, of them 1.5 for Q, 2.4 for the merge; over 131072 positions of 32 heads 246 (92 for
// the bytes; steps of 16 positions, one block of 8 warps per SM). Two blocks of 8 warps
// per SM with up to 16 rows (one of 8: 29 us; one of 16: 25.2 where this was 25.2, and
// 26.2 with its warps held to within two steps of one another, so that no block is done
// early); with 32 rows the outputs take the registers of one.
//
// Numbers: cached values are exact in f16 (kv4.cuh). Queries are brought to f16
// by a power of two per row that puts the row's largest value into
// [2^14, 2^15): exact down to 2^-29 of it. Probabilities are f16 with the
// running maximum at 2^7 to 2^15 (rescaled only when the maximum grows by more
// than 2^8), so that those below 2^-21 of the largest still have 11 bits. Sums,
// maxima and outputs are f32.
#include "kv4_attn.cuh"
#include "sm100.cuh"
#include "timeline.cuh"

namespace fdl {

namespace {

constexpr int A4_WARPS = 8, A4_THREADS = A4_WARPS * 32;
constexpr int A4_CLUSTER = 8;                // splits that join on chip

// c += A (16 x 16, rows) * B (16 x 8, columns), f16 with f32 sums.
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t* a, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void lds(const uint8_t* p, uint32_t (&r)[4]) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    r[0] = v.x;
    r[1] = v.y;
    r[2] = v.z;
    r[3] = v.w;
}
__device__ __forceinline__ void lds(const uint8_t* p, uint32_t (&r)[2]) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r[0] = v.x;
    r[1] = v.y;
}
__device__ __forceinline__ void lds(const uint8_t* p, uint32_t (&r)[1]) {
    r[0] = *reinterpret_cast<const uint32_t*>(p);
}

template <int D, int MT>
struct A4 {
    static constexpr int KS = MT == 1 ? 32 : 16;                 // positions per step of a warp
    static constexpr int OCC = MT == 1 ? 2 : 1;                  // blocks per SM
    static constexpr int STAGES = OCC == 2 ? 64 / KS : 96 / KS;  // of a warp's ring
    static constexpr int CB = D / 2, SB = D / KV4_GROUP;         // bytes of a row
    static constexpr int KK = D / 16;                            // k-steps of S
    static constexpr int NT = KS / 8;                            // 8-column tiles of S
    static constexpr int ND = D / 8;                             // 8-column tiles of O
    static constexpr int ROWS = 16 * MT;
    static constexpr int OFF_K = 0, OFF_V = KS * CB, OFF_KS = 2 * KS * CB,
                         OFF_VS = OFF_KS + KS * SB;
    static constexpr int STAGE = OFF_VS + KS * SB;
    static constexpr int RING = A4_WARPS * STAGES * STAGE;
    // after the steps the ring holds the warps' outputs, rows of D + 4 floats
    static constexpr int PROW = D + 4;
    static constexpr int PART = A4_WARPS * ROWS * PROW * 4;
    static constexpr int OFF_Q = RING > PART ? RING : PART;      // Q fragments
    static constexpr int OFF_RS = OFF_Q + MT * KK * 512;         // row scales
    static constexpr int OFF_ML = OFF_RS + ROWS * 4;             // warps' (max, sum)
    // the cluster's partial rows of the rows that this block joins: D + 4 floats
    // (output, maximum, sum) from each split, ROWS / cluster rows rounded up
    static constexpr int RROW = (D + 4) * 4;
    static constexpr int OFF_BAR = OFF_ML + A4_WARPS * ROWS * 8;
    static constexpr int OFF_RCV = OFF_BAR + 16;
    static constexpr int TOTAL = OFF_RCV + (ROWS + A4_CLUSTER) * RROW;
    static_assert(TOTAL <= (OCC == 2 ? 113 : 227) * 1024, "shared memory");
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
__global__ void __launch_bounds__(A4_THREADS, A4<D, MT>::OCC)
kv4_attn_kernel(const Kv4AttnArgs a) {
    using S = A4<D, MT>;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sb = sm100::smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    // block -> (sequence, kv head, row chunk, split)
    int u = blockIdx.x;
    const int split = u % a.n_splits;
    const int unit = u / a.n_splits;
    u = unit;
    const int chunk = u % a.chunks;
    u /= a.chunks;
    const int h = u % a.Hkv, bb = u / a.Hkv;
    const int row0 = chunk * a.chunk_rows;

    const int rank = split % a.cluster;
    const int own = min(a.chunk_rows, a.rows - row0);                 // rows that exist
    const int mine_rows = (own + a.cluster - 1 - rank) / a.cluster;   // rows rank, rank + cluster..
    const uint32_t bar = sb + S::OFF_BAR;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::OFF_BAR + 8);
    if (a.cluster > 1 && threadIdx.x == 0) {
        *abort_flag = 0;
        sm100::mbar_init(bar, 1);
        sm100::fence_barrier_init();
        // every split of the cluster sends a row of D + 2 floats for each of them
        sm100::mbar_arrive_expect_tx(bar, (uint32_t)(a.cluster * mine_rows * (D * 4 + 8)));
    }
    if (threadIdx.x == 0) FDL_TL(0, 0);
    pdl_wait();
    pdl_trigger();
    if (threadIdx.x == 0) FDL_TL(0, 1);

    // Q: row r of the chunk by warp r % 8, D / 32 dims per lane (all loads first)
    uint32_t qw[2 * MT][D / 64];
#pragma unroll
    for (int x = 0; x < 2 * MT; ++x) {
        const int pr = row0 + warp + x * A4_WARPS;
#pragma unroll
        for (int k = 0; k < D / 64; ++k) qw[x][k] = 0;
        if (pr < a.rows) {
            const bf16* src = a.q + RowAt(a, h, pr).at(a, bb, D) + lane * (D / 32);
            if constexpr (D == 128) {
                const uint2 v = *reinterpret_cast<const uint2*>(src);
                qw[x][0] = v.x;
                qw[x][1] = v.y;
            } else {
                qw[x][0] = *reinterpret_cast<const uint32_t*>(src);
            }
        }
    }

    const Seen seen(a, bb);
    // this split's run of indexes, whole steps but for the last
    const int steps_all = (seen.count + S::KS - 1) / S::KS;
    const int sps = (steps_all + a.n_splits - 1) / a.n_splits;
    const int i0 = min(split * sps, steps_all) * S::KS;
    const int i1 = min(seen.count, i0 + sps * S::KS);
    const int n_steps = i1 > i0 ? (i1 - i0 + S::KS - 1) / S::KS : 0;
    const int mine = n_steps > warp ? (n_steps - warp + A4_WARPS - 1) / A4_WARPS : 0;

    const size_t head = ((size_t)bb * a.Hkv + h) * a.L;
    const uint8_t* kc = a.k + head * S::CB;
    const uint8_t* vc = a.v + head * S::CB;
    const uint8_t* ks = a.ks + head * S::SB;
    const uint8_t* vs = a.vs + head * S::SB;
    const uint32_t ring = warp * (S::STAGES * S::STAGE);

    auto request = [&](int n) {              // the n-th step of this warp
        if (n < mine) {
            const uint32_t st = sb + ring + (n % S::STAGES) * S::STAGE;
            const int base = i0 + (warp + n * A4_WARPS) * S::KS;
            constexpr int CH = S::CB / 16, RX = 32 / CH;         // pieces of a row, rows at once
            const int r0 = lane / CH, ch = lane % CH;
            // the halves of a row swapped on every second pair of rows
            const uint32_t to = st + r0 * S::CB + ((CH == 4 ? ch ^ (r0 & 2) : ch) << 4);
            if (base + S::KS <= i1 && (base >= seen.first || base + S::KS <= seen.first)) {
                // one run of positions, all there
                const size_t p0 = base >= seen.first ? base + seen.gap : base;
                const uint8_t* ksrc = kc + p0 * S::CB + lane * 16;
                const uint8_t* vsrc = vc + p0 * S::CB + lane * 16;
#pragma unroll
                for (int x = 0; x < S::KS / RX; ++x) {
                    cp_async<16>(to + S::OFF_K + x * RX * S::CB, ksrc + x * RX * S::CB, true);
                    cp_async<16>(to + S::OFF_V + x * RX * S::CB, vsrc + x * RX * S::CB, true);
                }
                if constexpr (S::KS == 32) {
                    const size_t at = (p0 + lane) * S::SB;
                    cp_async<S::SB>(st + S::OFF_KS + lane * S::SB, ks + at, true);
                    cp_async<S::SB>(st + S::OFF_VS + lane * S::SB, vs + at, true);
                } else {                     // K's scales by half of the lanes, V's by the other
                    const size_t at = (p0 + (lane & 15)) * S::SB;
                    cp_async<S::SB>(st + S::OFF_KS + lane * S::SB, (lane < 16 ? ks : vs) + at,
                                    true);
                }
            } else {
#pragma unroll
                for (int x = 0; x < S::KS / RX; ++x) {
                    const int i = base + r0 + x * RX;
                    const bool there = i < i1;
                    const size_t off = (size_t)(there ? seen.pos(i) : 0) * S::CB + ch * 16;
                    cp_async<16>(to + S::OFF_K + x * RX * S::CB, kc + off, there);
                    cp_async<16>(to + S::OFF_V + x * RX * S::CB, vc + off, there);
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int row = S::KS == 32 ? lane : lane & 15, i = base + row;
                    const bool there = i < i1;
                    const size_t off = (size_t)(there ? seen.pos(i) : 0) * S::SB;
                    if (S::KS == 32 || (lane >> 4) == x)
                        cp_async<S::SB>(st + (x ? S::OFF_VS : S::OFF_KS) + row * S::SB,
                                        (x ? vs : ks) + off, there);
                }
            }
        }
        cp_commit();                         // empty groups keep the count
    };
#pragma unroll
    for (int n = 0; n < S::STAGES - 1; ++n) request(n);

    // Q fragments: word (mt, kk, lane (g, t), w) holds row mt*16 + g + 8*(w & 1),
    // dims D/4 t + 4 kk + 2 (w >> 1), +1.
#pragma unroll
    for (int x = 0; x < 2 * MT; ++x) {
        const int r = warp + x * A4_WARPS;
        float v[D / 32];
        uint32_t mb = 0;
#pragma unroll
        for (int k = 0; k < D / 64; ++k) {
            v[2 * k] = __uint_as_float(qw[x][k] << 16);
            v[2 * k + 1] = __uint_as_float(qw[x][k] & 0xffff0000u);
            mb = bf16x2_max_abs(mb, qw[x][k]);
        }
        mb = __reduce_max_sync(0xffffffffu, bf16x2_max_bits(mb));
        float f, inv;
        kv4_row_scale(mb, &f, &inv);
        if (lane == 0)
            reinterpret_cast<float*>(smem + S::OFF_RS)[r] = kv4_score_scale(a.scale_log2, inv);
#pragma unroll
        for (int k = 0; k < D / 64; ++k) {
            const int d = lane * (D / 32) + 2 * k;                // this pair's first dim
            const int qt = d / (D / 4), in = d % (D / 4);
            const int kk = in >> 2, w = ((r >> 3) & 1) | ((in >> 1) & 1) << 1;
            const int at = (((r >> 4) * S::KK + kk) * 32 + (r & 7) * 4 + qt) * 4 + w;
            reinterpret_cast<uint32_t*>(smem + S::OFF_Q)[at] =
                pack_half2(v[2 * k] * f, v[2 * k + 1] * f);
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) FDL_TL(0, 2);

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
        cp_wait<S::STAGES - 2>();
        if (n == 0 && threadIdx.x == 0) FDL_TL(0, 3);
        __syncwarp();                        // the step is there, the last one's stage free
        request(n + S::STAGES - 1);
        const uint8_t* st = smem + ring + (n % S::STAGES) * S::STAGE;
        const int base = i0 + (warp + n * A4_WARPS) * S::KS;

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
                const uint8_t* ka = st + S::OFF_K + row * S::CB;
                if constexpr (D == 128) {
                    lds(ka + ((t ^ (row & 2)) << 4), kw[nt]);
                    sc[nt] = *reinterpret_cast<const uint16_t*>(st + S::OFF_KS + row * S::SB +
                                                                2 * t);
                } else {
                    lds(ka + 8 * t, kw[nt]);
                    sc[nt] = st[S::OFF_KS + row * S::SB + t] * 0x0101u;
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
                        lds(smem + S::OFF_Q + ((mt * S::KK + 2 * w + x) * 32 + lane) * 16,
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
        if (base + S::KS > i1) {
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
                mx[mt][x] = v;
                grow |= (v - m[mt][x]) * rs[mt][x] > 8.f;
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
                    const float alpha =
                        mn == -INFINITY ? 1.f : kv4_weight(m[mt][x], mn, rs[mt][x]);
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
                const float base_m = kv4_base(m[mt][x]);
#pragma unroll
                for (int nt = 0; nt < S::NT; ++nt) {
                    const float2 e = kv4_exponents(s[mt][nt][2 * x], s[mt][nt][2 * x + 1], base_m,
                                                   rs[mt][x]);
                    const float p0 = ex2(e.x), p1 = ex2(e.y);
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
                    const uint8_t* va = st + S::OFF_V + row * S::CB;
                    if constexpr (D == 128) {
                        lds(va + ((((g >> 1) ^ (row & 2)) << 4) | ((g & 1) << 3)), vw[x][e]);
                        sc[e] = st[S::OFF_VS + row * S::SB + g];
                    } else {
                        lds(va + 4 * g, vw[x][e]);
                        sc[e] = st[S::OFF_VS + row * S::SB + (g >> 1)];
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
    if (threadIdx.x == 0) FDL_TL(0, 4);

    // ---- the warps' outputs joined in shared memory
    if (a.cluster > 1) sm100::cluster_arrive();                  // its barrier is set up
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            l[mt][x] += __shfl_xor_sync(0xffffffffu, l[mt][x], 1);
            l[mt][x] += __shfl_xor_sync(0xffffffffu, l[mt][x], 2);
        }
    __syncthreads();                         // every warp has left its ring
    const int live = min(A4_WARPS, n_steps); // warps that took a step
    float2* ml = reinterpret_cast<float2*>(smem + S::OFF_ML);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int r = mt * 16 + g + 8 * x;
            if (t == 0) ml[warp * S::ROWS + r] = make_float2(m[mt][x], l[mt][x]);
            if (r >= own || warp >= live) continue;
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
        }
    if (a.cluster > 1) sm100::cluster_wait();
    __syncthreads();
    if (threadIdx.x == 0) FDL_TL(0, 5);
    const float* row_scale = reinterpret_cast<const float*>(smem + S::OFF_RS);
    // row r, columns [4c, 4c + 4): out, to the workspace, or to the block that joins r
    auto finish = [&](int r, int c, float4 v, float M, float sum) {
        if (a.parts > 1) {
            const size_t at = ((size_t)unit * a.parts + split / a.cluster) * a.chunk_rows + r;
            *reinterpret_cast<float4*>(a.part + at * D + 4 * c) = v;
            if (c == 0) a.part_ml[at] = make_float4(M, sum, row_scale[r], 0.f);
            return;
        }
        const RowAt row(a, h, row0 + r);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;          // nothing visible: 0
        __nv_bfloat162 lo = __floats2bfloat162_rn(v.x * inv, v.y * inv);
        __nv_bfloat162 hi = __floats2bfloat162_rn(v.z * inv, v.w * inv);
        *reinterpret_cast<uint2*>(a.out + row.at(a, bb, D) + 4 * c) =
            make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
        if (a.lse && c == 0) a.lse[row.lse(a, bb)] = kv4_lse(M, row_scale[r], sum);
    };
    for (int it = threadIdx.x; it < own * (D / 4); it += A4_THREADS) {
        const int r = it / (D / 4), c = it % (D / 4);
        float2 p[A4_WARPS];
        float4 v[A4_WARPS];
        float M = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < A4_WARPS; ++w) {
            p[w] = ml[w * S::ROWS + r];      // (-inf, 0) of a warp without a step
            v[w] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (w < live)
                v[w] = reinterpret_cast<const float4*>(
                    reinterpret_cast<const float*>(smem) +
                    (size_t)(w * S::ROWS + r) * S::PROW)[slot(c)];
            M = fmaxf(M, p[w].x);
        }
        const float Ms = kv4_base(M), scale = row_scale[r];
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < A4_WARPS; ++w) {
            const float f = kv4_weight(p[w].x, Ms, scale);
            sum += p[w].y * f;
            acc.x += v[w].x * f;
            acc.y += v[w].y * f;
            acc.z += v[w].z * f;
            acc.w += v[w].w * f;
        }
        if (a.cluster == 1) {
            finish(r, c, acc, M, sum);
        } else {
            const int to = r % a.cluster, at = (r / a.cluster) * a.cluster + rank;
            const uint32_t dst = sm100::cluster_map(sb + S::OFF_RCV + at * S::RROW, to);
            const uint32_t rb = sm100::cluster_map(bar, to);
            sm100::st_async_f4(dst + 16 * c, acc, rb);
            if (c == 0) sm100::st_async_f2(dst + D * 4, make_float2(M, sum), rb);
        }
    }
    if (a.cluster > 1) {
        // ---- the rows that this block joins, once every split has sent them
        const bool got = a.polled ? sm100::mbar_poll(bar, 0, abort_flag, a.err)
                                  : sm100::mbar_wait(bar, 0, abort_flag, a.err);
        for (int it = threadIdx.x; got && it < mine_rows * (D / 4); it += A4_THREADS) {
            const int k = it / (D / 4), c = it % (D / 4), r = k * a.cluster + rank;
            float M = -INFINITY, sum = 0.f;
            float2 p[A4_CLUSTER];
            float4 v[A4_CLUSTER];
#pragma unroll
            for (int x = 0; x < A4_CLUSTER; ++x)
                if (x < a.cluster) {
                    const uint8_t* row = smem + S::OFF_RCV + (k * a.cluster + x) * S::RROW;
                    p[x] = *reinterpret_cast<const float2*>(row + D * 4);
                    v[x] = reinterpret_cast<const float4*>(row)[c];
                    M = fmaxf(M, p[x].x);
                }
            const float Ms = kv4_base(M), scale = row_scale[r];
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int x = 0; x < A4_CLUSTER; ++x)
                if (x < a.cluster) {
                    const float f = kv4_weight(p[x].x, Ms, scale);
                    sum += p[x].y * f;
                    acc.x += v[x].x * f;
                    acc.y += v[x].y * f;
                    acc.z += v[x].z * f;
                    acc.w += v[x].w * f;
                }
            finish(r, c, acc, M, sum);
        }
        if (!got) {
            // Nothing may land in a block that left: the others have sent their rows once
            // each of their threads has come here too or left, and what was sent lands.
            // (An arrival of every block's, waited for by all of them: 0.2 us more.)
            sm100::cluster_arrive();
            sm100::cluster_wait();
            sm100::mbar_wait_drain(bar, 0, a.err);
        }
    }
    if (threadIdx.x == 0) FDL_TL(0, 6);
}

template <int D, int MT>
int capacity(int c) {
    static std::atomic<int> known[9];
    return kv4_clusters((const void*)kv4_attn_kernel<D, MT>, A4_THREADS, A4<D, MT>::TOTAL, c,
                        known);
}

template <int D, int MT>
cudaError_t run_a4(const Kv4AttnArgs& a, long long units, cudaStream_t st) {
    using S = A4<D, MT>;
    auto kfn = kv4_attn_kernel<D, MT>;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = kv4_allow_smem(kfn, S::TOTAL, allowed);
    if (e != cudaSuccess) return e;
    return launch_pdl(kfn, dim3((unsigned)(units * a.n_splits)), dim3(A4_THREADS), S::TOTAL, st,
                      a.cluster, a);
}

}  // namespace

int kv4_few_clusters(int head_dim, int mt, int c) {
    if (head_dim == 128) return mt == 1 ? capacity<128, 1>(c) : capacity<128, 2>(c);
    return mt == 1 ? capacity<64, 1>(c) : capacity<64, 2>(c);
}

cudaError_t launch_kv4_attn_few(const Kv4AttnArgs& a, const Kv4Plan& p, int head_dim,
                                cudaStream_t st) {
    if (head_dim == 128)
        return p.mt == 1 ? run_a4<128, 1>(a, p.units, st) : run_a4<128, 2>(a, p.units, st);
    return p.mt == 1 ? run_a4<64, 1>(a, p.units, st) : run_a4<64, 2>(a, p.units, st);
}

}  // namespace fdl

FDL_TL_READER(fdl_timeline_kv4_attention)
