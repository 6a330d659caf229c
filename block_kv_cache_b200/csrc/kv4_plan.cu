// Attention over the 4-bit K/V cache: which kernel, how many splits, and the
// kernel that joins partial results.
#include "kv4_attn.cuh"
#include "timeline.cuh"

namespace fdl {

namespace {

// The partial outputs of a row joined: one block per row of a unit, a warp taking
// every 8th part and a lane D / 32 columns. A warp has its own maximum, so that all
// loads go out at once; the warps are joined in shared memory.
constexpr int JOIN_WARPS = 8;

template <int D>
__global__ void __launch_bounds__(32 * JOIN_WARPS) kv4_join_kernel(const Kv4AttnArgs a) {
    __shared__ float part[JOIN_WARPS][D];
    __shared__ float2 ml[JOIN_WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int chunk = blockIdx.x % a.chunks, u = blockIdx.x / a.chunks;
    const int h = u % a.Hkv, bb = u / a.Hkv;
    const int r = blockIdx.y, pr = chunk * a.chunk_rows + r;
    if (threadIdx.x == 0) FDL_TL(0, 0);
    pdl_wait();
    pdl_trigger();
    if (threadIdx.x == 0) FDL_TL(0, 1);
    if (pr >= a.rows) return;
    const size_t at = (size_t)blockIdx.x * a.parts * a.chunk_rows + r;
    constexpr int E = D / 32, U = 5;         // columns per lane, parts at a time
    float acc[E], M = -INFINITY, sum = 0.f;
#pragma unroll
    for (int x = 0; x < E; ++x) acc[x] = 0.f;
    const float rs = a.part_ml[at].z;
    for (int s0 = warp; s0 < a.parts; s0 += U * JOIN_WARPS) {
        float2 p[U];
        float v[U][E];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int s = s0 + k * JOIN_WARPS;
            p[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int x = 0; x < E; ++x) v[k][x] = 0.f;
            if (s < a.parts) {
                const size_t i = at + (size_t)s * a.chunk_rows;
                p[k] = *reinterpret_cast<const float2*>(a.part_ml + i);
                const float2* src = reinterpret_cast<const float2*>(a.part + i * D + lane * E);
#pragma unroll
                for (int x = 0; x < E; x += 2) {
                    const float2 w = src[x / 2];
                    v[k][x] = w.x;
                    v[k][x + 1] = w.y;
                }
            }
        }
        float mn = M;
#pragma unroll
        for (int k = 0; k < U; ++k) mn = fmaxf(mn, p[k].x);
        const float ms = kv4_base(mn), f0 = kv4_weight(M, ms, rs);
        sum *= f0;
#pragma unroll
        for (int x = 0; x < E; ++x) acc[x] *= f0;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const float f = kv4_weight(p[k].x, ms, rs);
            sum += p[k].y * f;
#pragma unroll
            for (int x = 0; x < E; ++x) acc[x] += v[k][x] * f;
        }
        M = mn;
    }
#pragma unroll
    for (int x = 0; x < E; ++x) part[warp][lane * E + x] = acc[x];
    if (lane == 0) ml[warp] = make_float2(M, sum);
    __syncthreads();
    if (threadIdx.x >= D / 2) return;
    float2 w8[JOIN_WARPS];
    M = -INFINITY;
#pragma unroll
    for (int w = 0; w < JOIN_WARPS; ++w) {
        w8[w] = ml[w];
        M = fmaxf(M, w8[w].x);
    }
    const float Ms = kv4_base(M);
    float o0 = 0.f, o1 = 0.f;
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < JOIN_WARPS; ++w) {
        const float f = kv4_weight(w8[w].x, Ms, rs);
        o0 += part[w][2 * threadIdx.x] * f;
        o1 += part[w][2 * threadIdx.x + 1] * f;
        sum += w8[w].y * f;
    }
    const RowAt row(a, h, pr);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;              // nothing visible: 0
    *reinterpret_cast<__nv_bfloat162*>(a.out + row.at(a, bb, D) + 2 * threadIdx.x) =
        __floats2bfloat162_rn(o0 * inv, o1 * inv);
    if (a.lse && threadIdx.x == 0) a.lse[row.lse(a, bb)] = kv4_lse(M, rs, sum);
    if (threadIdx.x == 0) FDL_TL(0, 2);
}

// The most positions that a sequence may see.
int most_seen(const Kv4Attn& s) {
    if (s.sinks >= s.win_lo) return s.sinks > s.win_hi ? s.sinks : s.win_hi;
    return s.sinks + s.win_hi - s.win_lo;
}

int parts_of(const Kv4Plan& p) { return p.n_splits / p.cluster; }

}  // namespace

Kv4Plan kv4_attention_plan(const Kv4Attn& s, int sm_count) {
    Kv4Plan p;
    const int rows = s.block_len * (s.n_q_heads / s.n_kv_heads), seen = most_seen(s);
    // The tcgen05 kernel has the longer first and last parts. It is used where the 32-row
    // blocks of the other would not all run at once, or have much to do: positions times
    // blocks per SM beyond an edge that depends on the tiles of rows and the head size.
    // us, tcgen05 and the other:
    //   one block per unit (up to 32 rows), never: 32 heads of 128 over 2048 positions
    //     14.1 and 10.8, over 131072 300 and 245; heads of 64 276 and 166
    //   more blocks than SMs: 40 units of 128 rows x 128 over 1024 13.7 and 26.9, 24 of
    //     224 over 256 12.5 and 13.9; the worst there is, 160 units of 40 rows x 64, one
    //     more round of blocks on 148 SMs, over 1024 28.0 and 25.3
    //   128 rows x 128, edge 850: 32 units over 900 (778) 12.9 and 13.4, over 1200 (1038)
    //     13.7 and 15.8; 8 units over 2048 (443) 15.5 and 10.6, over 5200 (1124) 17.9 and
    //     17.4, over 6000 18.5 and 18.8
    //   256 rows x 128, edge 1850: 8 units of 224 over 4096 (1550) 23.8 and 22.8, over 5000
    //     (1892) 25.0 and 26.4; 16 of 256 over 2048 (1771) 30.5 and 21.8, 16 of 224 over
    //     3000 (2270) 30.4 and 29.2, over 4096 32.5 and 36.9
    //   128 rows x 64, edge 1500: 32 units over 1200 (1038) 11.3 and 10.3, over 1800 (1557)
    //     12.7 and 13.6; 8 units over 6000 (1297) 15.3 and 12.7, over 10000 (2162) 17.1
    //     and 17.8
    //   256 rows x 64, edge 2600: 8 units of 224 over 6000 (2270) 21.5 and 20.4, over 8000
    //     (3027) 22.3 and 25.5; 16 units over 3000 (2270) 24.5 and 19.5, over 5000 (3784)
    //     28.3 and 29.5
    const long long blocks = (long long)s.batch * s.n_kv_heads * ((rows + 31) / 32);
    const long long edge = s.head_dim == 128 ? (rows <= 128 ? 850 : 1850)
                                             : (rows <= 128 ? 1500 : 2600);
    p.many = rows > 32 && (blocks > sm_count || blocks * seen > edge * sm_count);
    if (p.many) {
        p.chunks = (rows + 255) / 256;
        p.chunk_rows = (rows + p.chunks - 1) / p.chunks;
        p.mt = p.chunk_rows <= 128 ? 1 : 2;
    } else {
        p.mt = rows <= 16 ? 1 : 2;
        p.chunks = (rows + 16 * p.mt - 1) / (16 * p.mt);
        p.chunk_rows = (rows + p.chunks - 1) / p.chunks;
    }
    p.units = (long long)s.batch * s.n_kv_heads * p.chunks;
    // as many splits as fill the GPU once, each of 64 (few rows) or 128 positions
    const int slots = sm_count * (!p.many && p.mt == 1 ? 2 : 1), least = p.many ? 128 : 64;
    long long n = p.units < slots ? slots / p.units : 1;
    const long long most = (seen + least - 1) / least;
    if (n > most) n = most;
    if (n < 1) n = 1;
    auto clusters = [&](int c) {
        return p.many ? kv4_many_clusters(s.head_dim, p.mt, c)
                      : kv4_few_clusters(s.head_dim, p.mt, c);
    };
    // Many splits: clusters of 2, which leave no SM out, and partial results of each
    // (a token over 131072 positions of 4 kv heads: 25.8 us; of 4: 27.9, of 8: 28.4).
    if (n > 8) {
        const long long fit = clusters(2) / p.units, want = n / 2;
        p.cluster = 2;
        p.n_splits = 2 * (int)(fit > 0 && fit < want ? fit : want);
        return p;
    }
    // fewer while the clusters would not all be resident at once
    for (; n > 1; --n) {
        const int fit = clusters((int)n);
        if (fit <= 0 || p.units <= fit) break;
    }
    p.cluster = p.n_splits = (int)n;
    return p;
}

int kv4_clusters(const void* kernel, int threads, size_t smem, int c, std::atomic<int>* known) {
    const int n0 = known[c].load(std::memory_order_relaxed);
    if (n0 > 0) return n0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(c);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = c;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    known[c].store(n, std::memory_order_relaxed);
    return n;
}

void kv4_attention_warm() {
    for (int d = 64; d <= 128; d += 64)
        for (int mt = 1; mt <= 2; ++mt)
            for (int c = 2; c <= 8; ++c) {
                (void)kv4_few_clusters(d, mt, c);
                (void)kv4_many_clusters(d, mt, c);
            }
}

size_t kv4_attention_workspace_bytes(const Kv4Attn& s, const Kv4Plan& p) {
    if (parts_of(p) == 1) return 16;
    return (size_t)p.units * parts_of(p) * p.chunk_rows * (s.head_dim * 4 + 16);
}

cudaError_t launch_kv4_attention(const Kv4Attn& s, const Kv4Plan& p, const void* q,
                                 const Kv4Ptrs& c, void* out, float* lse, void* ws, int* err,
                                 cudaStream_t st) {
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
    a.by_g = FastDiv((uint32_t)a.G);
    a.L = s.seq_len;
    a.rows = a.B * a.G;
    a.chunks = p.chunks;
    a.chunk_rows = p.chunk_rows;
    a.n_splits = p.n_splits;
    a.cluster = p.cluster;
    a.parts = parts_of(p);
    a.sinks = s.sinks;
    a.win_lo = s.win_lo;
    a.win_hi = s.win_hi;
    a.scale_log2 = fminf(s.scale * 1.4426950408889634f, 3.4028234663852886e38f);
    a.polled = s.polled;
    a.err = err;
    a.part = (float*)ws;
    a.part_ml = (float4*)((float*)ws + (size_t)p.units * a.parts * a.chunk_rows * s.head_dim);
    cudaError_t e = p.many ? launch_kv4_attn_many(a, p, s.head_dim, st)
                           : launch_kv4_attn_few(a, p, s.head_dim, st);
    if (e != cudaSuccess || a.parts == 1) return e;
    const dim3 grid((unsigned)p.units, p.chunk_rows), block(32 * JOIN_WARPS);
    return s.head_dim == 128 ? launch_pdl(kv4_join_kernel<128>, grid, block, 0, st, 0, a)
                             : launch_pdl(kv4_join_kernel<64>, grid, block, 0, st, 0, a);
}

}  // namespace fdl

FDL_TL_READER(fdl_timeline_kv4_join)
