// Block attention over the 4-bit K/V cache, many query rows per kv head, on the
// 5th-generation tensor cores.
//
// A block of threads owns up to 128 MT packed query rows (the 128 TMEM lanes of
// one or two MMA tiles) and a run of visible positions, taken in tiles of 64:
//   S = Q K^T       Q and K in shared memory
//   O += P V        P in TMEM, in place of the scores it came from
// The warps divide the work by kind, a tile moving from one to the next:
//   6 conversion warps: codes and scales from memory into registers (PF pieces of 16
//       positions ahead; positions behind the end as zeros: code 0 under scale 0),
//       then K and V as f16 into a ring of STAGES operand tiles; a cached value is
//       converted once per block, for all its rows
//   2 matrix warps, one per softmax warpgroup: tcgen05.mma as soon as the operands are
//       there (one thread for both took 0.5 us per product of a tile and held
//       everything else up)
//   2 softmax warpgroups, a thread per row: each runs its own online softmax, with
//       its own S buffers and O. With two MMA tiles a warpgroup has the rows of
//       one; with one tile both have all rows and take every second tile of
//       positions, and their outputs are joined on the way out of TMEM.
// A warp's scores of the next tile are computed while it works on this one. 16 warps,
// so that a thread may have 128 registers; a scheduler has two softmax warps and two
// of the others.
//
// What bounds it, in us:
//   32 sequences, 32 queries of 28 heads on 4 kv heads of 128, 1024 positions: 24.4
//     (9.3 for the products at the measured 1615 TFLOP/s, 2.9 for the bytes). 3.5
//     before the first scores (Q's rows, their powers of two; 1.5 before that for the
//     launch), 16 tiles at 1.0 each, 2.3 for the output. A tile: two softmax warps on a
//     scheduler take 1450 cycles when nothing else issues (measured alone), the
//     conversion's share of it is 500 more.
//   8 sequences, 32 queries of 32 heads on 8, a window of 1060 positions: 15.6, two
//     blocks of 128 rows each: 3.0 before the first scores, 5.9 for 9 tiles, 5.0 for
//     the output and the join.
// The 128 registers do not hold all of three forms (heads and tiles: 64, 1 spills 32
// bytes, 64, 2 4, 128, 1 28).
// The first and last parts run once through fresh instructions, so they are kept
// short: a row of Q comes as one bulk copy (16 bytes per lane with cp.async: first
// scores 1.1 later), a row's output leaves TMEM as bf16 and the block as one bulk copy
// per row (4.9 -> 2.5 with the stores 8 bytes per lane), and the weights of a join are
// found by the lanes of one warp (3.0 -> 2.4; rows pushed to the block that joins them
// with st.async: 2.6 for the pushes alone). Measured and not kept: four conversion warps
// (28.2 and 18.2), K and V converted by different warps (26.2 and 17.3) or their
// pieces in turn (25.7 and 16.6); the search for the next tile's maximum beside this
// one's exponentials (1.5 more).
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
constexpr int M4_SOFT = 8, M4_CONV = 6;      // softmax and conversion warps
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

// A run of bytes (multiples of 16) from shared to global memory, and their arrival.
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, int bytes) {
    asm volatile(
        "cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n\t"
        "cp.async.bulk.commit_group;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}
// From global to shared memory, counted on a barrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, int bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
            "r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}
__device__ __forceinline__ void bulk_store_wait() {
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

template <int D, int MT>
struct M4 {
    static constexpr int CB = D / 2, SB = D / KV4_GROUP;         // bytes of a cached row
    static constexpr int DC = D / 64;                            // 128-byte columns of a row
    static constexpr int STAGES = MT == 2 ? 4 : 5;               // of operand tiles
    static constexpr int PF = 3;                                 // pieces of codes in registers
    static constexpr int KV = DC * M4_KT * 128;                  // an f16 K or V tile
    static constexpr int QC = 128 * 128;                         // 64 dims of 128 rows
    static constexpr int OFF_Q = 0;                              // [MT][DC][128 rows][128 B]
    static constexpr int OFF_K = OFF_Q + MT * DC * QC, OFF_V = OFF_K + STAGES * KV;
    static constexpr int OFF_ML = OFF_V + STAGES * KV;           // float2 per row
    static constexpr int OFF_BAR = OFF_ML + 256 * 8;
    static constexpr int TOTAL = 1024 + OFF_BAR + 512;
    // after the tiles, the output in their place: bf16 rows OROW bytes apart (the next
    // row's banks are 4 further), or, for a cluster, [128 MT][D] f32 with the 16-byte
    // pieces swapped by row, and the rows' (max, sum, score scale) in Q's place
    static constexpr int OFF_O = OFF_K, OROW = D * 2 + 16;
    static_assert(MT * 128 * D * 4 <= OFF_ML - OFF_K && MT * 128 * 16 <= MT * DC * QC, "output");
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
    auto kv_full = [&](int t) { return bars + 8 * (t % ST); };
    auto kv_free = [&](int t) { return bars + 64 + 8 * (t % ST); };
    auto kv_ph = [](int t) { return (uint32_t)(t / ST) & 1u; };
    // a warpgroup's j-th tile: scores there, probabilities there, O has taken them
    auto s_full = [&](int w, int j) { return bars + 128 + 16 * w + 8 * (j & 1); };
    auto p_full = [&](int w, int j) { return bars + 160 + 16 * w + 8 * (j & 1); };
    auto o_done = [&](int w, int j) { return bars + 192 + 16 * w + 8 * (j & 1); };
    auto ph = [](int j) { return (uint32_t)(j >> 1) & 1u; };
    const uint32_t q_full = bars + 224, all_done = bars + 232;
    auto q_in = [&](int i) { return bars + 256 + 8 * i; };       // 32 rows of Q as they are
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
            mbar_init(kv_full(t), 4);
            mbar_init(kv_free(t), MT);
        }
        for (int w = 0; w < 2; ++w)
            for (int j = 0; j < 2; ++j) {
                mbar_init(s_full(w, j), 1);
                mbar_init(p_full(w, j), 4);
                mbar_init(o_done(w, j), 1);
            }
        mbar_init(q_full, M4_SOFT);
        for (int i = 0; i < 4 * MT; ++i) mbar_init(q_in(i), 1);
        mbar_init(all_done, 2);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == M4_MMA_WARP) tmem_alloc(smem_u32(tmem_slot), S::TMEM);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // where the row of Q lies that this thread fetches
    const bf16* q_at = nullptr;
    if (warp < 4 * MT && warp * 32 + lane < own)
        q_at = a.q + RowAt(a, h, row0 + warp * 32 + lane).at(a, bb, D);
    pdl_wait();
    pdl_trigger();
    if (warp < 4 * MT) {
        if (lane == 0) mbar_arrive_expect_tx(q_in(warp), max(0, min(32, own - warp * 32)) * D * 2);
        __syncwarp();
        if (q_at)
            bulk_load(sb + S::OFF_Q + (warp * 32 + lane) * (D * 2), q_at, D * 2, q_in(warp));
    }
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
    if (warp >= M4_SOFT && warp < M4_MMA_WARP) {
        // ------------------------------------------------------------ conversion
        // Pieces of 16 positions, four to a tile, dealt to the warps in turn; a thread
        // has 32 dims (16 bytes of codes, two groups) of one or two of them. Lanes are
        // dealt so that 8 of them store to different banks.
        constexpr int XN = S::DC;
        const int cw = warp - M4_SOFT, pieces_all = 4 * nt;
        const int key0 = D == 128 ? ((lane >> 1) & 3) + 4 * (lane >> 4) : lane >> 1;
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
        auto load = [&](int n, Raw& r) {     // piece n, of tile n / 4
#pragma unroll
            for (int x = 0; x < XN; ++x) {
                const int i = i0 + 16 * n + key0 + 8 * x;
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
        auto convert = [&](int n, const uint4 (&c)[XN], const uint32_t (&scale)[XN], uint32_t off) {
#pragma unroll
            for (int x = 0; x < XN; ++x) {
                const int key = 16 * (n & 3) + key0 + 8 * x;
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
        };
        Raw raw[S::PF];
#pragma unroll
        for (int p = 0; p < S::PF; ++p)
            if (cw + p * M4_CONV < pieces_all) load(cw + p * M4_CONV, raw[p]);
        for (int n0 = cw; ok && n0 < pieces_all; n0 += S::PF * M4_CONV) {
#pragma unroll
            for (int p = 0; p < S::PF; ++p) {
                const int n = n0 + p * M4_CONV, t = n >> 2;
                if (!ok || n >= pieces_all) break;
                if (!(ok = mbar_wait_warp(kv_free(t), kv_ph(t) ^ 1u, abort_flag, a.err))) break;
                convert(n, raw[p].k, raw[p].ks, S::OFF_K + (t % ST) * S::KV);
                convert(n, raw[p].v, raw[p].vs, S::OFF_V + (t % ST) * S::KV);
                fence_proxy_async();         // the matrix instructions read it
                __syncwarp();
                if (lane == 0) mbar_arrive(kv_full(t));
                if (n + S::PF * M4_CONV < pieces_all) load(n + S::PF * M4_CONV, raw[p]);
            }
        }
    } else if (warp >= M4_MMA_WARP) {
        // ------------------------------------------------------------ products
        // The whole warp waits and counts, one lane issues: what is the same for the
        // warp stays in uniform registers, where the instructions take their operands.
        const int w = __shfl_sync(0xffffffffu, warp, 0) - M4_MMA_WARP;
        constexpr uint32_t id_s = idesc_f16(128, KT, false), id_o = idesc_f16(128, D, true);
        const int mine = tiles_of(w);
        // descriptors of the first k-step; the others are a few 16-byte units on
        const uint64_t q0 = umma_desc_sw128(sb + S::OFF_Q + (MT == 2 ? w * S::DC * S::QC : 0));
        const uint64_t k0 = umma_desc_sw128(sb + S::OFF_K);
        const uint64_t v0 = umma_desc_sw128_mn(sb + S::OFF_V, KT * 128);
        auto scores = [&](int j) {
            const int t = tile_of(w, j);
            // S buffer j & 1 holds P of tile j - 2 until O has taken it
            ok = mbar_wait_warp(kv_full(t), kv_ph(t), abort_flag, a.err) &&
                 mbar_wait_warp(o_done(w, j), ph(j) ^ 1u, abort_flag, a.err);
            if (!ok) return;
            tc_fence_after();
            const uint64_t kt = k0 + (uint64_t)((t % ST) * (S::KV >> 4));
            const uint32_t s_at = tmem + (2 * w + (j & 1)) * KT;
            if (lane == 0) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    umma_bf16(s_at, q0 + ((k >> 2) * (S::QC >> 4) + (k & 3) * 2),
                              kt + ((k >> 2) * (KT * 128 >> 4) + (k & 3) * 2), id_s, k > 0);
                umma_commit(s_full(w, j));
            }
            __syncwarp();
        };
        ok = mbar_wait_warp(q_full, 0, abort_flag, a.err);
        if (ok && mine > 0) scores(0);
        for (int j = 0; ok && j < mine; ++j) {
            if (j + 1 < mine) scores(j + 1);
            const int t = tile_of(w, j);
            ok = ok && mbar_wait_warp(p_full(w, j), ph(j), abort_flag, a.err);
            if (!ok) break;
            tc_fence_after();
            const uint64_t vt = v0 + (uint64_t)((t % ST) * (S::KV >> 4));
            const uint32_t p_at = tmem + (2 * w + (j & 1)) * KT;
            if (lane == 0) {
#pragma unroll
                for (int k = 0; k < KT / 16; ++k)
                    umma_f16_ts(tmem + S::TMEM_O + w * D, p_at + k * 8, vt + k * (2048 >> 4), id_o,
                                (j > 0 || k > 0) ? 1u : 0u);
                umma_commit(o_done(w, j));
                umma_commit(kv_free(t));
            }
            __syncwarp();
        }
        // whatever was issued ends before TMEM is given back
        if (lane == 0) umma_commit(all_done);
        __syncwarp();
        mbar_wait_drain(all_done, 0, a.err);
    } else {
        // ------------------------------------------------------------ softmax
        const int w = warp >> 2, q = warp & 3;
        const int lr = q * 32 + lane;                            // lane of the MMA tile
        const int r = (MT == 2 ? w * 128 : 0) + lr;
        const uint32_t lanes = (uint32_t)(q * 32) << 16;
        // Q: its rows are on their way, one after the other, into their place; a thread
        // takes its row (one tile: half of it, the other warpgroup has the rest) into
        // registers, finds its scale and stores it back as f16, in the 16-byte pieces
        // that the matrix instructions want swapped by row. The piece that lane l takes
        // k-th, k ^ 2 l in the field of 8 elements, makes both the reads (at a distance
        // of whole rows) and the writes (k ^ 2 l ^ l = k ^ 3 l) hit different banks.
        float rs;
        {
            uint8_t* q_sh = smem + S::OFF_Q + (MT == 2 ? w * S::DC * S::QC : 0);
            constexpr int NP = D / 8 / (3 - MT);
            const int l2 = ((lane << 1) ^ ((lane >> 2 & 1) * 11)) & 7;
            auto piece = [&](int k) {
                return (MT == 2 ? 0 : w * NP) + ((k & ~7) | (((k & 7) ^ l2) & (NP - 1)));
            };
            uint4 x[NP];
            uint32_t mb = 0;
            ok = mbar_wait_drain(q_in(MT == 2 ? warp : q), 0, a.err);
            ok = __all_sync(0xffffffffu, ok);
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                x[k] = make_uint4(0, 0, 0, 0);
                if (r < own)
                    x[k] = *reinterpret_cast<const uint4*>(q_sh + lr * (D * 2) + piece(k) * 16);
                mb = bf16x2_max_abs(bf16x2_max_abs(mb, x[k].x), x[k].y);
                mb = bf16x2_max_abs(bf16x2_max_abs(mb, x[k].z), x[k].w);
            }
            mb = bf16x2_max_bits(mb);
            if constexpr (MT == 1) {
                uint32_t* halves = reinterpret_cast<uint32_t*>(smem + S::OFF_ML);
                halves[128 * w + lr] = mb;
                bar_sync(1, 32 * M4_SOFT);
                mb = max(mb, halves[128 * (w ^ 1) + lr]);
            } else {
                bar_sync(2 + w, 128);        // the warpgroup has read its rows
            }
            float f, inv;
            kv4_row_scale(mb, &f, &inv);
            rs = kv4_score_scale(a.scale_log2, inv);
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const uint32_t v[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
                uint32_t b[4];
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    b[y] = pack_half2(__uint_as_float(v[y] << 16) * f,
                                      __uint_as_float(v[y] & 0xffff0000u) * f);
                const int p = piece(k);
                *reinterpret_cast<uint4*>(q_sh + (p >> 3) * S::QC + lr * 128 +
                                          (((p & 7) ^ (lr & 7)) << 4)) =
                    make_uint4(b[0], b[1], b[2], b[3]);
            }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
        if (threadIdx.x == 0) FDL_TL(0, 2);

        float m = -INFINITY, l = 0.f;
        const int mine = tiles_of(w);
        // warps whose rows are all padding only keep the barriers going
        const bool live = (MT == 2 ? w * 128 : 0) + q * 32 < own;
        for (int j = 0; ok && j < mine; ++j) {
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
                const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                if (__any_sync(0xffffffffu, (mx - m) * rs > 8.f)) {
                    const float mn = fmaxf(m, mx);
                    // nothing seen so far: l and O are zero and stay so
                    const float alpha = mn == -INFINITY ? 1.f : kv4_weight(m, mn, rs);
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
                const float base_m = kv4_base(m);
                float l2[2] = {0.f, 0.f};
#pragma unroll
                for (int c0 = 0; c0 < KT; c0 += 32) {
                    uint32_t pk[16];
#pragma unroll
                    for (int c = 0; c < 32; c += 2) {
                        const float2 e = kv4_exponents(s[c0 + c], s[c0 + c + 1], base_m, rs);
                        const float p0 = ex2(e.x), p1 = ex2(e.y);
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

        // ---- outputs, in TMEM: a thread takes its row, or, with one tile of rows, half
        // of its columns, from both warpgroups' halves of the positions
        float2* ml = reinterpret_cast<float2*>(smem + S::OFF_ML);
        if (MT == 1) ml[128 * w + lr] = make_float2(m, l);
        bar_sync(1, 32 * M4_SOFT);           // all tiles have been read
        float f[2] = {1.f, 1.f};             // what either half is multiplied with
        if constexpr (MT == 1) {
            const float2 p0 = ml[lr], p1 = ml[128 + lr];
            m = fmaxf(p0.x, p1.x);
            const float ms = kv4_base(m);
            f[0] = kv4_weight(p0.x, ms, rs);
            f[1] = kv4_weight(p1.x, ms, rs);
            l = p0.y * f[0] + p1.y * f[1];
        }
        if (a.cluster == 1) {
            const float inv = l == 0.f ? 0.f : 1.f / l;          // nothing visible: 0
            f[0] *= inv;
            f[1] *= inv;
        }
        constexpr int NC = MT == 2 ? D : D / 2;                  // columns of a thread
        const int c0 = MT == 2 ? 0 : w * NC;
        const uint32_t o_at = tmem + lanes + S::TMEM_O + (MT == 2 ? w * D : c0);
#pragma unroll 2
        for (int c = 0; c < NC; c += 16) {
            float o[16], y[16];
#pragma unroll
            for (int x = 0; x < 16; ++x) o[x] = y[x] = 0.f;
            // an accumulator that no tile went into holds anything
            if (tiles_of(MT == 2 ? w : 0) > 0) tmem_ld<16>(o_at + c, o);
            if (MT == 1 && tiles_of(1) > 0) tmem_ld<16>(o_at + D + c, y);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 16; ++x) o[x] = MT == 2 ? o[x] * f[0] : o[x] * f[0] + y[x] * f[1];
            if (a.cluster == 1) {
                uint32_t b[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const __nv_bfloat162 t = __floats2bfloat162_rn(o[2 * x], o[2 * x + 1]);
                    b[x] = *reinterpret_cast<const uint32_t*>(&t);
                }
                uint4* to = reinterpret_cast<uint4*>(smem + S::OFF_O + r * S::OROW + (c0 + c) * 2);
                to[0] = make_uint4(b[0], b[1], b[2], b[3]);
                to[1] = make_uint4(b[4], b[5], b[6], b[7]);
            } else {
                float4* to = reinterpret_cast<float4*>(smem + S::OFF_O) + r * (D / 4);
#pragma unroll
                for (int x = 0; x < 16; x += 4)
                    to[((c0 + c + x) >> 2) ^ (lr & 7)] =
                        make_float4(o[x], o[x + 1], o[x + 2], o[x + 3]);
            }
        }
        if (a.cluster == 1) {
            // a row's bytes lie together here and in the output: one copy by its thread
            fence_proxy_async();
            if (MT == 1) bar_sync(1, 32 * M4_SOFT);
            if ((MT == 2 || w == 0) && r < own) {
                const RowAt row(a, h, row0 + r);
                bulk_store(a.out + row.at(a, bb, D), sb + S::OFF_O + r * S::OROW, D * 2);
                if (a.lse) a.lse[row.lse(a, bb)] = kv4_lse(m, rs, l);
                bulk_store_wait();
            }
        } else if (MT == 2 || w == 0) {
            reinterpret_cast<float4*>(smem + S::OFF_Q)[r] = make_float4(m, l, rs, 0.f);
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
        // cluster, ..., four at a time to a warp, D / 4 lanes each
        cluster_sync();
        constexpr int LR = D / 4, RX = 32 / LR, NX = 4 / RX;     // lanes of a row, rows at once
        const int rank = split % a.cluster, c4 = lane % LR;
        const int mine_rows = (own + a.cluster - 1 - rank) / a.cluster;
        for (int kb = warp * 4; kb < mine_rows; kb += M4_THREADS / 32 * 4) {
            // the first two splits' columns, on their way while the weights are found
            float4 v[2][NX];
            auto fetch = [&](int c) {
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int x = 0; x < NX; ++x) {
                        const int k = kb + x * RX + lane / LR;
                        const int row = min(k, mine_rows - 1) * a.cluster + rank;
                        v[y][x] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (c + y < a.cluster)
                            v[y][x] = ld_cluster_f4(cluster_map(
                                sb + S::OFF_O + (row * (D / 4) + (c4 ^ (row & 7))) * 16, c + y));
                    }
            };
            // lane 8 i + c: what split c's part of row kb + i is multiplied with
            const int k = kb + (lane >> 3), c = lane & 7, r = k * a.cluster + rank;
            float4 p = make_float4(-INFINITY, 0.f, 0.f, 0.f);
            if (k < mine_rows && c < a.cluster)
                p = ld_cluster_f4(cluster_map(sb + S::OFF_Q + r * 16, c));
            fetch(0);
            float M = p.x;
#pragma unroll
            for (int o = 1; o < 8; o *= 2) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
            // of a split that is not there: 0
            float wt = c < a.cluster ? kv4_weight(p.x, kv4_base(M), p.z) : 0.f, sum = p.y * wt;
#pragma unroll
            for (int o = 1; o < 8; o *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            unsigned long long to = 0;       // where the row goes
            if (k < mine_rows) {
                if (a.parts > 1) {
                    const size_t at =
                        ((size_t)unit * a.parts + split / a.cluster) * a.chunk_rows + r;
                    to = reinterpret_cast<unsigned long long>(a.part + at * D);
                    if (c == 0) a.part_ml[at] = make_float4(M, sum, p.z, 0.f);
                } else {
                    const RowAt row(a, h, row0 + r);
                    to = reinterpret_cast<unsigned long long>(a.out + row.at(a, bb, D));
                    wt *= sum == 0.f ? 0.f : 1.f / sum;          // nothing visible: 0
                    if (a.lse && c == 0) a.lse[row.lse(a, bb)] = kv4_lse(M, p.z, sum);
                }
            }
            __syncwarp();
            float4 acc[NX];
#pragma unroll
            for (int x = 0; x < NX; ++x) acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int c0 = 0;;) {
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int x = 0; x < NX; ++x) {
                        // of a split that is not there: 0
                        const float f = __shfl_sync(0xffffffffu, wt,
                                                    8 * (x * RX + lane / LR) + ((c0 + y) & 7));
                        acc[x].x += v[y][x].x * f;
                        acc[x].y += v[y][x].y * f;
                        acc[x].z += v[y][x].z * f;
                        acc[x].w += v[y][x].w * f;
                    }
                c0 += 2;
                if (c0 >= a.cluster) break;
                fetch(c0);
            }
#pragma unroll
            for (int x = 0; x < NX; ++x) {
                const unsigned long long at =
                    __shfl_sync(0xffffffffu, to, 8 * (x * RX + lane / LR));
                if (!at) continue;
                if (a.parts > 1) {
                    reinterpret_cast<float4*>(at)[c4] = acc[x];
                } else {
                    const __nv_bfloat162 lo = __floats2bfloat162_rn(acc[x].x, acc[x].y);
                    const __nv_bfloat162 hi = __floats2bfloat162_rn(acc[x].z, acc[x].w);
                    reinterpret_cast<uint2*>(at)[c4] =
                        make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                   *reinterpret_cast<const uint32_t*>(&hi));
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
