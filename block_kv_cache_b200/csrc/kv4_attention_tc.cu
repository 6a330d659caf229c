// Block attention over the 4-bit K/V cache, many query rows per kv head, on the
// 5th-generation tensor cores.
//
// A block of threads owns up to 128 MT packed query rows (the 128 TMEM lanes of
// one or two MMA tiles) and a run of visible positions, taken in tiles of 64:
//   S = Q K^T       Q and K in shared memory
//   O += P V        P in TMEM, in place of the scores it came from
// The warps divide the work by kind, a tile moving from one to the next:
//   4 conversion warps: codes and scales from memory into registers (PF tiles
//       ahead; positions behind the end as zeros: code 0 under scale 0), then K and
//       V as f16 into a ring of STAGES operand tiles; a cached value is converted
//       once per block, for all its rows
//   2 matrix warps (one thread each, one per softmax warpgroup): tcgen05.mma as soon
//       as the operands are there (one thread for both took 0.5 us per product
//       of a tile and held everything else up)
//   2 softmax warpgroups, a thread per row: each runs its own online softmax, with
//       its own S buffers and O. With two MMA tiles a warpgroup has the rows of
//       one; with one tile both have all rows and take every second tile of
//       positions, and join their outputs at the end.
// A warp's scores of the next tile are computed while it works on this one.
//
// What bounds it: 32 sequences, 32 queries of 28 heads on 4 kv heads of 128, 1024
// positions: 28.2 us (9.3 for the products at the measured 1615 TFLOP/s, 2.9 for the
// bytes). A block's 8 tiles per split take 1.1 us each: the exponentials, maxima and
// conversions of two softmax warps per scheduler (1450 cycles when nothing else
// issues, measured alone) beside the conversion warps. The rest is 4.7 us before the
// first scores (start, Q) and 3.8 after the last (join, output). Searching the next
// tile's maximum beside this one's exponentials took 29.5 us, one matrix warp for
// both warpgroups 37.9. 8 sequences of 32 queries of 32 heads on 8 over a window of
// 1060 positions: 18.2 us, of which the loop is a third.
//
// Numbers as in kv4_attention.cu: f16 operands (cached values exact, queries by a
// power of two per row), f32 scores, sums and outputs, f16 probabilities at 2^7 to
// 2^15 at the running maximum, which is raised when it grows by more than 2^8.
#include "kv4_attn.cuh"
#include "sm100.cuh"
#include "timeline.cuh"

namespace fdl {

namespace {

constexpr int M4_KT = 64;                    // positions per tile
constexpr int M4_SOFT = 8, M4_CONV = 4;      // softmax and conversion warps
constexpr int M4_MMA_WARP = M4_SOFT + M4_CONV;
constexpr int M4_THREADS = 32 * (M4_MMA_WARP + 2);

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float* f) {
    uint32_t* r = reinterpret_cast<uint32_t*>(f);
#pragma unroll
    for (int c = 0; c < N; c += 16)
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, "
            "%10, %11, %12, %13, %14, %15}, [%16];"
            : "=r"(r[c]), "=r"(r[c + 1]), "=r"(r[c + 2]), "=r"(r[c + 3]), "=r"(r[c + 4]),
              "=r"(r[c + 5]), "=r"(r[c + 6]), "=r"(r[c + 7]), "=r"(r[c + 8]), "=r"(r[c + 9]),
              "=r"(r[c + 10]), "=r"(r[c + 11]), "=r"(r[c + 12]), "=r"(r[c + 13]),
              "=r"(r[c + 14]), "=r"(r[c + 15])
            : "r"(taddr + c)
            : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, "
        "%10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void bar_sync(int id, int n) {
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}

// f16 x f16 -> f32, A [M x K], B [N x K]; b_mn: B lies with N contiguous.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn) {
    return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}

// D (+)= A B with A in TMEM: lane = row, two f16 of K per column.
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

template <int D, int MT>
struct M4 {
    static constexpr int CB = D / 2, SB = D / KV4_GROUP;         // bytes of a cached row
    static constexpr int DC = D / 64;                            // 128-byte columns of a row
    static constexpr int STAGES = 4;
    static constexpr int PF = 3;                                 // tiles of codes in registers
    static constexpr int KV = DC * M4_KT * 128;                  // an f16 K or V tile
    static constexpr int QC = 128 * 128;                         // 64 dims of 128 rows
    static constexpr int OFF_Q = 0;                              // [MT][DC][128 rows][128 B]
    static constexpr int OFF_K = OFF_Q + MT * DC * QC, OFF_V = OFF_K + STAGES * KV;
    static constexpr int OFF_ML = OFF_V + STAGES * KV;           // float2 per row
    static constexpr int OFF_BAR = OFF_ML + 256 * 8;
    static constexpr int TOTAL = 1024 + OFF_BAR + 512;
    // after the tiles, the output: [256][D] f32, 16-byte pieces swapped by row (with
    // one tile of rows, of either warpgroup's positions), and weights in Q's place
    static constexpr int OFF_O = OFF_K;
    static_assert(256 * D * 4 <= OFF_ML - OFF_K && 8 * 256 * 4 <= MT * DC * QC, "output");
    static_assert(TOTAL <= 227 * 1024, "shared memory");
    static constexpr uint32_t TMEM_O = 4 * M4_KT;                // S: [warpgroup][2] of 64
    static constexpr uint32_t TMEM = 512;
};

// Timeline events (timeline builds): 0 entry, 1 after the dependency wait, 2 Q in
// place, 3 first scores, 4 last probabilities, 5 outputs complete, 6 exit.
template <int D, int MT>
__global__ void __launch_bounds__(M4_THREADS, 1)
kv4_attn_tc_kernel(const Kv4AttnArgs a) {
    using namespace sm100;
    using S = M4<D, MT>;
    constexpr int KT = M4_KT, ST = S::STAGES;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_at = smem_u32(smem_raw), pad = (1024u - (raw_at & 1023u)) & 1023u;
    uint8_t* smem = smem_raw + pad;
    const uint32_t sb = raw_at + pad;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t bars = sb + S::OFF_BAR;
    auto k_full = [&](int t) { return bars + 8 * (t % ST); };
    auto v_full = [&](int t) { return bars + 32 + 8 * (t % ST); };
    auto k_free = [&](int t) { return bars + 64 + 8 * (t % ST); };
    auto v_free = [&](int t) { return bars + 96 + 8 * (t % ST); };
    auto kv_ph = [](int t) { return (uint32_t)(t / ST) & 1u; };
    // a warpgroup's j-th tile: scores there, probabilities there, O has taken them
    auto s_full = [&](int w, int j) { return bars + 128 + 16 * w + 8 * (j & 1); };
    auto p_full = [&](int w, int j) { return bars + 160 + 16 * w + 8 * (j & 1); };
    auto o_done = [&](int w, int j) { return bars + 192 + 16 * w + 8 * (j & 1); };
    auto ph = [](int j) { return (uint32_t)(j >> 1) & 1u; };
    const uint32_t q_full = bars + 224, all_done = bars + 232;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::OFF_BAR + 240);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    // block -> (sequence, kv head, row chunk, split)
    int u = blockIdx.x;
    const int split = u % a.n_splits;
    const int unit = u / a.n_splits;
    u = unit;
    const int chunk = u % a.chunks;
    u /= a.chunks;
    const int h = u % a.Hkv, bb = u / a.Hkv;
    const int row0 = chunk * a.chunk_rows, own = min(a.chunk_rows, a.rows - row0);

    if (threadIdx.x == 0) {
        FDL_TL(0, 0);
        for (int t = 0; t < ST; ++t) {
            mbar_init(k_full(t), M4_CONV);
            mbar_init(v_full(t), M4_CONV);
            mbar_init(k_free(t), MT);
            mbar_init(v_free(t), MT);
        }
        for (int w = 0; w < 2; ++w)
            for (int j = 0; j < 2; ++j) {
                mbar_init(s_full(w, j), 1);
                mbar_init(p_full(w, j), 4);
                mbar_init(o_done(w, j), 1);
            }
        mbar_init(q_full, M4_SOFT);
        mbar_init(all_done, 2);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == M4_MMA_WARP) tmem_alloc(smem_u32(tmem_slot), S::TMEM);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_trigger();
    if (threadIdx.x == 0) FDL_TL(0, 1);

    const Seen seen(a, bb);
    // this split's run of indexes, in pieces of 16
    const int pieces = (seen.count + 15) / 16;
    const int per = (pieces + a.n_splits - 1) / a.n_splits;
    const int i0 = min(split * per, pieces) * 16;
    const int i1 = min(seen.count, i0 + per * 16);
    const int nt = i1 > i0 ? (i1 - i0 + KT - 1) / KT : 0;
    // warpgroup w's tiles: all, or every second one from the w-th on
    auto tiles_of = [&](int w) { return MT == 2 ? nt : (nt + 1 - w) / 2; };
    auto tile_of = [&](int w, int j) { return MT == 2 ? j : 2 * j + w; };
    bool ok = true;
    // four columns of a finished row, rounded once
    auto store4 = [&](bf16* at, float4 v, float inv) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x * inv, v.y * inv);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(v.z * inv, v.w * inv);
        *reinterpret_cast<uint2*>(at) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                       *reinterpret_cast<const uint32_t*>(&hi));
    };

    if (warp >= M4_SOFT && warp < M4_MMA_WARP) {
        // ------------------------------------------------------------ conversion
        // 16 positions per warp and tile; a thread has 32 dims (16 bytes of codes,
        // two groups) of one or two of them. Lanes are dealt so that 8 of them
        // store to different banks.
        constexpr int XN = S::DC;
        const int cw = warp - M4_SOFT;
        const int key0 = 16 * cw + (D == 128 ? ((lane >> 1) & 3) + 4 * (lane >> 4) : lane >> 1);
        const int ch = D == 128 ? (lane & 1) + 2 * ((lane >> 3) & 1) : lane & 1;
        const size_t head = ((size_t)bb * a.Hkv + h) * a.L;
        const uint8_t* kc = a.k + head * S::CB + ch * 16;
        const uint8_t* vc = a.v + head * S::CB + ch * 16;
        const uint8_t* ks = a.ks + head * S::SB + ch * 2;
        const uint8_t* vs = a.vs + head * S::SB + ch * 2;
        struct Raw {
            uint4 k[XN], v[XN];
            uint32_t ks[XN], vs[XN];
        };
        auto load = [&](int t, Raw& r) {
#pragma unroll
            for (int x = 0; x < XN; ++x) {
                const int i = i0 + t * KT + key0 + 8 * x;
                r.k[x] = r.v[x] = make_uint4(0, 0, 0, 0);
                r.ks[x] = r.vs[x] = 0;
                if (i < i1) {
                    const size_t pos = seen.pos(i);
                    r.k[x] = __ldcg(reinterpret_cast<const uint4*>(kc + pos * S::CB));
                    r.ks[x] = __ldcg(reinterpret_cast<const uint16_t*>(ks + pos * S::SB));
                    r.v[x] = __ldcg(reinterpret_cast<const uint4*>(vc + pos * S::CB));
                    r.vs[x] = __ldcg(reinterpret_cast<const uint16_t*>(vs + pos * S::SB));
                }
            }
        };
        // f16 tile: [64-dim column][position][128 bytes], 16-byte pieces swapped by position
        auto convert = [&](const uint4 (&c)[XN], const uint32_t (&scale)[XN], uint32_t off) {
#pragma unroll
            for (int x = 0; x < XN; ++x) {
                const int key = key0 + 8 * x;
                uint8_t* dst = smem + off + (ch >> 1) * (KT * 128) + key * 128;
                const uint32_t s2 = e4m3x2_half2(scale[x]);
                const uint32_t w[4] = {c[x].x, c[x].y, c[x].z, c[x].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t b[4];
                    e2m1x8_half2(w[i], b);
                    const uint32_t s = __byte_perm(s2, 0, i < 2 ? 0x1010 : 0x3232);
#pragma unroll
                    for (int y = 0; y < 4; ++y) b[y] = hmul2(b[y], s);
                    const int piece = (ch & 1) * 4 + i;
                    *reinterpret_cast<uint4*>(dst + ((piece ^ (key & 7)) << 4)) =
                        make_uint4(b[0], b[1], b[2], b[3]);
                }
            }
            fence_proxy_async();             // the matrix instructions read it
            __syncwarp();
        };
        Raw raw[S::PF];
#pragma unroll
        for (int p = 0; p < S::PF; ++p)
            if (p < nt) load(p, raw[p]);
        for (int t0 = 0; ok && t0 < nt; t0 += S::PF) {
#pragma unroll
            for (int p = 0; p < S::PF; ++p) {
                const int t = t0 + p;
                if (!ok || t >= nt) break;
                if (!(ok = mbar_wait_warp(k_free(t), kv_ph(t) ^ 1u, abort_flag, a.err))) break;
                convert(raw[p].k, raw[p].ks, S::OFF_K + (t % ST) * S::KV);
                if (lane == 0) mbar_arrive(k_full(t));
                if (!(ok = mbar_wait_warp(v_free(t), kv_ph(t) ^ 1u, abort_flag, a.err))) break;
                convert(raw[p].v, raw[p].vs, S::OFF_V + (t % ST) * S::KV);
                if (lane == 0) mbar_arrive(v_full(t));
                if (t + S::PF < nt) load(t + S::PF, raw[p]);
            }
        }
    } else if (warp >= M4_MMA_WARP) {
        // ------------------------------------------------------------ products
        const int w = warp - M4_MMA_WARP;
        if (lane == 0) {
            constexpr uint32_t id_s = idesc_f16(128, KT, false), id_o = idesc_f16(128, D, true);
            const int mine = tiles_of(w);
            // descriptors of the first k-step; the others are a few 16-byte units on
            const uint64_t q0 = umma_desc_sw128(sb + S::OFF_Q + (MT == 2 ? w * S::DC * S::QC : 0));
            const uint64_t k0 = umma_desc_sw128(sb + S::OFF_K);
            const uint64_t v0 = umma_desc_sw128_mn(sb + S::OFF_V, KT * 128);
            auto scores = [&](int j) {
                const int t = tile_of(w, j);
                // S buffer j & 1 holds P of tile j - 2 until O has taken it
                ok = mbar_wait(k_full(t), kv_ph(t), abort_flag, a.err) &&
                     mbar_wait(o_done(w, j), ph(j) ^ 1u, abort_flag, a.err);
                if (!ok) return;
                tc_fence_after();
                const uint64_t kt = k0 + (uint64_t)((t % ST) * (S::KV >> 4));
                const uint32_t s_at = tmem + (2 * w + (j & 1)) * KT;
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    umma_bf16(s_at, q0 + ((k >> 2) * (S::QC >> 4) + (k & 3) * 2),
                              kt + ((k >> 2) * (KT * 128 >> 4) + (k & 3) * 2), id_s, k > 0);
                umma_commit(s_full(w, j));
                umma_commit(k_free(t));
            };
            ok = mbar_wait(q_full, 0, abort_flag, a.err);
            if (ok && mine > 0) scores(0);
            for (int j = 0; ok && j < mine; ++j) {
                if (j + 1 < mine) scores(j + 1);
                const int t = tile_of(w, j);
                ok = ok && mbar_wait(v_full(t), kv_ph(t), abort_flag, a.err) &&
                     mbar_wait(p_full(w, j), ph(j), abort_flag, a.err);
                if (!ok) break;
                tc_fence_after();
                const uint64_t vt = v0 + (uint64_t)((t % ST) * (S::KV >> 4));
                const uint32_t p_at = tmem + (2 * w + (j & 1)) * KT;
#pragma unroll
                for (int k = 0; k < KT / 16; ++k)
                    umma_f16_ts(tmem + S::TMEM_O + w * D, p_at + k * 8, vt + k * (2048 >> 4), id_o,
                                (j > 0 || k > 0) ? 1u : 0u);
                umma_commit(o_done(w, j));
                umma_commit(v_free(t));
            }
            // whatever was issued ends before TMEM is given back
            umma_commit(all_done);
            mbar_wait_drain(all_done, 0, a.err);
        }
    } else {
        // ------------------------------------------------------------ softmax
        const int w = warp >> 2, q = warp & 3;
        const int lr = q * 32 + lane;                            // lane of the MMA tile
        const int r = (MT == 2 ? w * 128 : 0) + lr;
        const uint32_t lanes = (uint32_t)(q * 32) << 16;
        // Q: rows into their places as they are, 16 bytes per lane; then a thread
        // takes its row, finds its scale and stores its half of the pieces (one
        // tile: the other warpgroup has the rest) or all, as f16 in place
        float rs;
        {
            constexpr int LR = D / 8, RX = 32 / LR;              // lanes of a row, rows at once
            constexpr int RW = MT == 2 ? 32 : 16;                // rows that this warp fetches
            uint8_t* q_sh = smem + S::OFF_Q + (MT == 2 ? w * S::DC * S::QC : 0);
            auto place = [&](int row, int i) {
                return (i >> 3) * S::QC + row * 128 + (((i & 7) ^ (row & 7)) << 4);
            };
            auto piece = [&](int row, int i) {
                return reinterpret_cast<uint4*>(q_sh + place(row, i));
            };
            // lane k knows where the warp's k-th row lies
            const int first = q * 32 + (MT == 2 ? 0 : 16 * w), i0q = lane % LR;
            const int mine = (MT == 2 ? w * 128 : 0) + first + lane;
            const bf16* at = mine < own && lane < RW
                                 ? a.q + RowAt(a, h, row0 + mine).at(a, bb, D) : nullptr;
#pragma unroll
            for (int k = 0; k < RW; k += RX) {
                const bf16* src = reinterpret_cast<const bf16*>(__shfl_sync(
                    0xffffffffu, reinterpret_cast<unsigned long long>(at), k + lane / LR));
                cp_async<16>(smem_u32(q_sh) + place(first + k + lane / LR, i0q),
                             src ? src + i0q * 8 : a.q, src != nullptr);
            }
            cp_commit();
            cp_wait<0>();
            if (MT == 2) __syncwarp();
            else bar_sync(1, 32 * M4_SOFT);
            uint32_t mb = 0;
#pragma unroll 8
            for (int i = 0; i < D / 8; ++i) {
                const uint4 x = *piece(lr, i);
                mb = bf16x2_max_abs(bf16x2_max_abs(mb, x.x), x.y);
                mb = bf16x2_max_abs(bf16x2_max_abs(mb, x.z), x.w);
            }
            mb = bf16x2_max_bits(mb);
            if (MT == 2) __syncwarp();
            else bar_sync(1, 32 * M4_SOFT);
            float f, inv;
            kv4_row_scale(mb, &f, &inv);
            rs = kv4_score_scale(a.scale_log2, inv);
#pragma unroll 4
            for (int k = 0; k < D / 8 / (3 - MT); ++k) {
                const int i = MT == 2 ? k : 2 * k + w;
                const uint4 x = *piece(lr, i);
                const uint32_t v[4] = {x.x, x.y, x.z, x.w};
                uint32_t b[4];
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    b[y] = pack_half2(__uint_as_float(v[y] << 16) * f,
                                      __uint_as_float(v[y] & 0xffff0000u) * f);
                *piece(lr, i) = make_uint4(b[0], b[1], b[2], b[3]);
            }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
        if (threadIdx.x == 0) FDL_TL(0, 2);

        float m = -INFINITY, l = 0.f;                            // log2 units
        const int mine = tiles_of(w);
        // warps whose rows are all padding only keep the barriers going
        const bool live = (MT == 2 ? w * 128 : 0) + q * 32 < own;
        for (int j = 0; j < mine; ++j) {
            if (!(ok = mbar_wait_warp(s_full(w, j), ph(j), abort_flag, a.err))) break;
            tc_fence_after();
            if (j == 0 && threadIdx.x == 0) FDL_TL(0, 3);
            if (live) {
                const uint32_t s_at = tmem + lanes + (2 * w + (j & 1)) * KT;
                float s[KT];
                tmem_ld<KT>(s_at, s);
                tmem_wait_ld();
                const int base = i0 + tile_of(w, j) * KT;
                if (base + KT > i1) {
#pragma unroll
                    for (int c = 0; c < KT; ++c)
                        if (base + c >= i1) s[c] = -INFINITY;
                }
                float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int c = 4; c < KT; ++c) m4[c & 3] = fmaxf(m4[c & 3], s[c]);
                const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * rs;
                if (__any_sync(0xffffffffu, mx > m + 8.f)) {
                    const float mn = fmaxf(m, mx);
                    // nothing seen so far: l and O are zero and stay so
                    const float alpha = mn == -INFINITY ? 1.f : ex2(m - mn);
                    m = mn;
                    l *= alpha;
                    if (j > 0) {
                        if (!(ok = mbar_wait_warp(o_done(w, j - 1), ph(j - 1), abort_flag, a.err)))
                            break;
                        tc_fence_after();
#pragma unroll
                        for (int c = 0; c < D; c += 16) {
                            float o[16];
                            const uint32_t at = tmem + lanes + S::TMEM_O + w * D + c;
                            tmem_ld<16>(at, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int x = 0; x < 16; ++x) o[x] *= alpha;
                            tmem_st16(at, reinterpret_cast<const uint32_t*>(o));
                        }
                    }
                }
                const float nm = m == -INFINITY ? 0.f : KV4_SHIFT - m;
                float l2[2] = {0.f, 0.f};
#pragma unroll
                for (int c0 = 0; c0 < KT; c0 += 32) {
                    uint32_t pk[16];
#pragma unroll
                    for (int c = 0; c < 32; c += 2) {
                        const float p0 = ex2(fmaf(s[c0 + c], rs, nm));
                        const float p1 = ex2(fmaf(s[c0 + c + 1], rs, nm));
                        l2[0] += p0;
                        l2[1] += p1;
                        pk[c >> 1] = pack_half2(p0, p1);
                    }
                    tmem_st16(s_at + (c0 >> 1), pk);
                }
                l += l2[0] + l2[1];
                tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full(w, j));
        }
        if (threadIdx.x == 0) FDL_TL(0, 4);
        if (ok && mine > 0)
            ok = mbar_wait_warp(o_done(w, mine - 1), ph(mine - 1), abort_flag, a.err);
        tc_fence_after();
        if (threadIdx.x == 0) FDL_TL(0, 5);

        // ---- outputs: a thread has a row, in TMEM; through shared memory (in the
        // tiles' place) to whole rows per warp
        const uint32_t o_at = tmem + lanes + S::TMEM_O + w * D;
        float4* orow = reinterpret_cast<float4*>(smem + S::OFF_O) + (w * 128 + lr) * (D / 4);
        float2* ml = reinterpret_cast<float2*>(smem + S::OFF_ML);
        // a row's last word, by its thread: its maximum and sum for the other splits,
        // or, of the only one, what its output is multiplied with
        auto settle = [&]() {
            if (a.cluster > 1) return make_float2(m, l);
            if (r < own && a.lse) a.lse[RowAt(a, h, row0 + r).lse(a, bb)] = kv4_lse(m, l);
            return make_float2(l == 0.f ? 0.f : 1.f / l, 0.f);   // nothing visible: 0
        };
        if (MT == 1) ml[128 * w + lr] = make_float2(m, l);
        bar_sync(1, 32 * M4_SOFT);           // all tiles have been read
        float f = 1.f;
        if constexpr (MT == 1) {
            // (max, sum) of the other warpgroup's half of the positions: both halves
            // under the common maximum
            const float2 other = ml[128 * (w ^ 1) + lr];
            const float mn = fmaxf(m, other.x), ms = mn == -INFINITY ? 0.f : mn;
            f = ex2(m - ms);
            l = l * f + other.y * ex2(other.x - ms);
            m = mn;
        }
#pragma unroll 4
        for (int c = 0; c < D; c += 16) {
            float o[16];
#pragma unroll
            for (int x = 0; x < 16; ++x) o[x] = 0.f;
            if (mine > 0) {
                tmem_ld<16>(o_at + c, o);
                tmem_wait_ld();
            }
#pragma unroll
            for (int x = 0; x < 16; x += 4)
                orow[((c + x) >> 2) ^ (lr & 7)] =
                    make_float4(o[x] * f, o[x + 1] * f, o[x + 2] * f, o[x + 3] * f);
        }
        if (MT == 1) bar_sync(1, 32 * M4_SOFT);
        if (MT == 2 || w == 0) ml[r] = settle();
        if (MT == 1) bar_sync(1, 32 * M4_SOFT);
        else __syncwarp();
        // row k of this warp, columns [4c, 4c + 4) for lane c; both halves' sum
        constexpr int LR = D / 4, RX = 32 / LR, RW = MT == 2 ? 32 : 16;
        const int first = MT == 2 ? w * 128 + q * 32 : warp * 16, c = lane % LR;
        float4* all = reinterpret_cast<float4*>(smem + S::OFF_O);
        auto fetch = [&](int row) {
            float4 v = all[row * (D / 4) + (c ^ (row & 7))];
            if constexpr (MT == 1) {
                const float4 y = all[(128 + row) * (D / 4) + (c ^ (row & 7))];
                v.x += y.x;
                v.y += y.y;
                v.z += y.z;
                v.w += y.w;
            }
            return v;
        };
        if (a.cluster == 1) {
            // lane k knows where the warp's k-th row goes
            const int row_k = first + lane;
            const unsigned long long at_k =
                lane < RW && row_k < own ? reinterpret_cast<unsigned long long>(
                                               a.out + RowAt(a, h, row0 + row_k).at(a, bb, D))
                                         : 0;
            const float inv_k = lane < RW ? ml[row_k].x : 0.f;
#pragma unroll 8
            for (int k = 0; k < RW; k += RX) {
                const int from = k + lane / LR;
                const unsigned long long at = __shfl_sync(0xffffffffu, at_k, from);
                const float inv = __shfl_sync(0xffffffffu, inv_k, from);
                const float4 v = fetch(first + from);
                if (at) store4(reinterpret_cast<bf16*>(at) + 4 * c, v, inv);
            }
        } else if constexpr (MT == 1) {
#pragma unroll 8
            for (int k = 0; k < RW; k += RX) {
                const int row = first + k + lane / LR;
                all[row * (D / 4) + (c ^ (row & 7))] = fetch(row);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == M4_MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, S::TMEM);
    }
    if (a.cluster > 1) {
        // ---- several splits, joined over the cluster: rank c takes rows c, c +
        // cluster, ... First what each split's part of them is multiplied with, a
        // thread per row; then the rows, D / 4 lanes each, all loads of UR at once.
        cluster_sync();
        constexpr int LR = D / 4, RX = 32 / LR, UR = 5;
        const int rank = split % a.cluster, c4 = lane % LR;
        const int mine_rows = (own + a.cluster - 1 - rank) / a.cluster;
        float* wt = reinterpret_cast<float*>(smem + S::OFF_Q);   // [8][256]
        for (int k = threadIdx.x; k < mine_rows; k += M4_THREADS) {
            const int row = k * a.cluster + rank;
            float2 p[8];
            float M = -INFINITY, sum = 0.f;
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (c < a.cluster) p[c] = ld_cluster_f2(cluster_map(sb + S::OFF_ML + row * 8, c));
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (c < a.cluster) M = fmaxf(M, p[c].x);
            const float Ms = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (c < a.cluster) {
                    p[c].x = ex2(p[c].x - Ms);
                    sum += p[c].y * p[c].x;
                }
            float inv = 1.f;
            if (a.parts > 1) {
                a.part_ml[((size_t)unit * a.parts + split / a.cluster) * a.chunk_rows + row] =
                    make_float2(M, sum);
            } else {
                inv = sum == 0.f ? 0.f : 1.f / sum;              // nothing visible: 0
                if (a.lse) a.lse[RowAt(a, h, row0 + row).lse(a, bb)] = kv4_lse(M, sum);
            }
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (c < a.cluster) wt[c * 256 + k] = p[c].x * inv;
        }
        __syncthreads();
        constexpr int KX = M4_THREADS / 32 * RX;                 // rows of the block at once
        for (int k0 = warp * RX + lane / LR; k0 < mine_rows; k0 += UR * KX) {
            float4 acc[UR];
#pragma unroll
            for (int x = 0; x < UR; ++x) acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int c = 0; c < a.cluster; c += 2) {
                float4 v[2][UR];
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int x = 0; x < UR; ++x) {
                        const int k = k0 + x * KX, row = k * a.cluster + rank;
                        if (c + y < a.cluster && k < mine_rows)
                            v[y][x] = ld_cluster_f4(cluster_map(
                                sb + S::OFF_O + (row * (D / 4) + (c4 ^ (row & 7))) * 16, c + y));
                    }
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int x = 0; x < UR; ++x) {
                        const int k = k0 + x * KX;
                        if (c + y < a.cluster && k < mine_rows) {
                            const float f = wt[(c + y) * 256 + k];
                            acc[x].x += v[y][x].x * f;
                            acc[x].y += v[y][x].y * f;
                            acc[x].z += v[y][x].z * f;
                            acc[x].w += v[y][x].w * f;
                        }
                    }
            }
#pragma unroll
            for (int x = 0; x < UR; ++x) {
                const int k = k0 + x * KX, row = k * a.cluster + rank;
                if (k >= mine_rows) continue;
                if (a.parts > 1) {
                    const size_t at =
                        ((size_t)unit * a.parts + split / a.cluster) * a.chunk_rows + row;
                    *reinterpret_cast<float4*>(a.part + at * D + 4 * c4) = acc[x];
                } else {
                    store4(a.out + RowAt(a, h, row0 + row).at(a, bb, D) + 4 * c4, acc[x], 1.f);
                }
            }
        }
        cluster_sync();                      // no block leaves while others read its memory
    }
    if (threadIdx.x == 0) FDL_TL(0, 6);
}

// Clusters of c blocks that the GPU holds at once, as for the other kernel.
template <int D, int MT>
int capacity(int c) {
    static std::atomic<int> known[9];
    return kv4_clusters((const void*)kv4_attn_tc_kernel<D, MT>, M4_THREADS, M4<D, MT>::TOTAL, c,
                        known);
}

template <int D, int MT>
cudaError_t run_m4(const Kv4AttnArgs& a, long long units, cudaStream_t st) {
    using S = M4<D, MT>;
    auto kfn = kv4_attn_tc_kernel<D, MT>;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = kv4_allow_smem(kfn, S::TOTAL, allowed);
    if (e != cudaSuccess) return e;
    return launch_pdl(kfn, dim3((unsigned)(units * a.n_splits)), dim3(M4_THREADS), S::TOTAL, st,
                      a.cluster, a);
}

}  // namespace

int kv4_many_clusters(int head_dim, int mt, int c) {
    if (head_dim == 128) return mt == 1 ? capacity<128, 1>(c) : capacity<128, 2>(c);
    return mt == 1 ? capacity<64, 1>(c) : capacity<64, 2>(c);
}

cudaError_t launch_kv4_attn_many(const Kv4AttnArgs& a, const Kv4Plan& p, int head_dim,
                                 cudaStream_t st) {
    if (head_dim == 128)
        return p.mt == 1 ? run_m4<128, 1>(a, p.units, st) : run_m4<128, 2>(a, p.units, st);
    return p.mt == 1 ? run_m4<64, 1>(a, p.units, st) : run_m4<64, 2>(a, p.units, st);
}

}  // namespace fdl

FDL_TL_READER(fdl_timeline_kv4_attention_tc)
