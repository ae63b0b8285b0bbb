// Single-query decode over a packed history: one new token per sequence attends, with
// exact softmax, the tokens of its routed 4-bit chunks and its bf16 local window.
//
// "Long-Context Fine-Tuning with Limited VRAM", technical summary section 2.1 (routed
// exact chunks next to a local window), with the history's values as packed.cuh defines
// them: z_t = q . k_t / sqrt(D), out = sum_t softmax(z)_t v_t.
//
// Bound by HBM, and at small batches by latency: a routed chunk is 72 D bytes (0.28 of
// bf16), read once for the G <= 8 query heads of its KV head.  The codes go from global
// memory straight into MMA operands, without shared memory: a warp takes a whole chunk,
// and the axes that the products contract or run along are permuted so that a lane's
// 16 (K) or 8 (V) bytes of a row are exactly its operand registers.  With lane = 4 r + c
// (r = lane / 4, c = lane % 4):
//   S^T = K Q^T   M = 16 tokens, N = 8 heads.  Row r of token tile t is token
//                 16 (r / 2) + 2 t + r % 2; lane c holds channels c D/4 .. + D/4, which
//                 the k index runs through two pairs at a time (the queries likewise).
//   O^T += V^T P^T  M = 16 channels, N = 8 heads.  Row r of channel tile u is channel
//                 (D/4) (r / 2) + 2 u + r % 2; lane c holds tokens 16 c .. + 16.  P, as
//                 S^T leaves it (tokens by heads), becomes that operand by one
//                 transposing move per 8 tokens.
// The tokens of the window go through the same products in pieces of 16, read as bf16.
//
// The units (routed chunks, then window pieces) of one (batch, KV head) are dealt to the
// warps of a thread-block cluster; every warp keeps its own running maximum, sum and
// output, which are merged through shared memory, first of the CTA, then of the
// cluster: one launch, no workspace, sums in a fixed order.
#include "packed.cuh"
#include "tc_ptx.cuh"

namespace hga {

namespace {

constexpr int CHK = 64;
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kPiece = 16;      // window tokens per unit
constexpr int kMaxRouted = 64;  // topk limit of the parameter check
constexpr int kHeads = 8;       // query heads per KV head: the N side of the products
constexpr int kMaxCluster = 8;  // portable cluster size
constexpr int kCtasPerSm = 2;

struct PackedDecodeArgs {
    const __nv_bfloat16 *q;
    const uint8_t *hist;
    const __nv_bfloat16 *kl;
    const __nv_bfloat16 *vl;
    const int32_t *idx;
    __nv_bfloat16 *out;
    float *lse;
    unsigned *status;
    long long cap, local_stride;
    int n_q_heads, n_kv_heads, topk, n_hist_chunks, n_local, n_cluster;
    float scale_log2;  // log2(e) / sqrt(D)
};

// Transposes the 8x8 b16 matrix of which lane 4 r + c holds (row r, columns 2 c, 2 c + 1).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// N bytes (a multiple of 8) of read-once data.
template <int N> __device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&w)[N / 4]) {
#pragma unroll
    for (int i = 0; i < N / 16; ++i) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p) + i);
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
    }
    if constexpr (N % 16 == 8) {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p + N / 16 * 16));
        w[N / 4 - 2] = v.x;
        w[N / 4 - 1] = v.y;
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) decode_packed_kernel(const PackedDecodeArgs a) {
    using P = Packed<D>;
    constexpr int NJ = D / 32;  // channel octets of a lane
    constexpr int NU = D / 8;   // 8-channel row tiles
    __shared__ int units[kMaxRouted];
    __shared__ int n_routed;
    __shared__ float wm[kWarps][kHeads], wl[kWarps][kHeads];
    __shared__ __align__(16) float wo[kWarps][kHeads][D + 4];
    __shared__ float cm[kHeads], cl[kHeads];        // the CTA's merged maximum and sum
    __shared__ __align__(16) float co[kHeads][D];   // and output

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = lane >> 2, c = lane & 3;
    const int G = a.n_q_heads / a.n_kv_heads;
    const int rank = (int)blockIdx.x % a.n_cluster;
    const int bg = (int)blockIdx.x / a.n_cluster;
    const int b = bg / a.n_kv_heads, g = bg % a.n_kv_heads;

    if (warp == 0) {  // the valid routes, in order; -1 is padding, anything else out of range is skipped
        const int32_t *sel = a.idx + (long long)bg * a.topk;
        int n = 0;
#pragma unroll
        for (int i0 = 0; i0 < kMaxRouted; i0 += 32) {
            const int j = i0 + lane < a.topk ? sel[i0 + lane] : -1;
            const bool ok = j >= 0 && j < a.n_hist_chunks;
            if (!ok && j != -1 && rank == 0) atomicOr(a.status, kDevBadIndex);
            const unsigned m = __ballot_sync(0xffffffffu, ok);
            if (ok) units[n + __popc(m & ((1u << lane) - 1u))] = j;
            n += __popc(m);
        }
        if (lane == 0) n_routed = n;
    }

    // queries of head r as the B operand: pair p of octet j of the lane's channels
    uint32_t qf[NJ][4];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (r < G)
            v = *reinterpret_cast<const uint4 *>(a.q + ((long long)b * a.n_q_heads + (long long)g * G + r) * D +
                                                 (D / 4) * c + 8 * j);
        qf[j][0] = v.x;
        qf[j][1] = v.y;
        qf[j][2] = v.z;
        qf[j][3] = v.w;
    }
    // state of heads 2c, 2c + 1: o[i] rows r (channel tile 2i) and r + 8 (tile 2i + 1)
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};  // l: this lane's tokens only
    float o[NU / 2][4];
#pragma unroll
    for (int i = 0; i < NU / 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    __syncthreads();

    const int nr = n_routed;
    const int n_units = nr + (a.n_local + kPiece - 1) / kPiece;
    const int step = a.n_cluster * kWarps;
    // a warp's units interleave over the CTAs first, so that few units use every SM
    int u = warp * a.n_cluster + rank;

    // one online-softmax step over NT tiles of 16 tokens: s holds raw scores of (token
    // rows r, r + 8; heads 2c, 2c + 1), -inf where masked; leaves P^T operands in pt
    auto softmax = [&](auto &s, auto &pt) {
        constexpr int NT = sizeof(s) / sizeof(s[0]);
        float corr[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float mx = fmaxf(s[0][h], s[0][2 + h]);
#pragma unroll
            for (int i = 1; i < NT; ++i) mx = fmaxf(mx, fmaxf(s[i][h], s[i][2 + h]));
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            const float m_new = fmaxf(m_run[h], mx * a.scale_log2);
            // a unit holds at least one unmasked token, so m_new is above -inf unless a
            // score is -inf or NaN; p must not become NaN for the -inf of a masked token
            const float m_sub = m_new == -INFINITY ? 0.f : m_new;
            corr[h] = exp2f(m_run[h] - m_sub);  // 0 at the first unit
            m_run[h] = m_new;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                s[i][h] = tc::ex2(fmaf(s[i][h], a.scale_log2, -m_sub));
                s[i][2 + h] = tc::ex2(fmaf(s[i][2 + h], a.scale_log2, -m_sub));
                sum += s[i][h] + s[i][2 + h];
            }
            l_run[h] = fmaf(l_run[h], corr[h], sum);
        }
        if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
            for (int i = 0; i < NU / 2; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][e] *= corr[e & 1];
        }
        // P is rounded to bf16 for the product, as in the other attention kernels
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            pt[2 * i] = transpose8(tc::pack_bf16(s[i][0], s[i][1]));
            pt[2 * i + 1] = transpose8(tc::pack_bf16(s[i][2], s[i][3]));
        }
    };

    for (; u < nr; u += step) {
        const uint8_t *rec = a.hist + ((long long)bg * a.cap + units[u]) * P::kRecord;
        const uint8_t *vrec = rec + P::kPart;
        uint32_t kw[8][NJ], vw[NU][2];
#pragma unroll
        for (int t = 0; t < 8; ++t)
            load_words<4 * NJ>(rec + (16 * (r >> 1) + 2 * t + (r & 1)) * (D / 2) + c * 4 * NJ, kw[t]);
#pragma unroll
        for (int i = 0; i < NU; ++i)
            load_words<8>(vrec + ((D / 4) * (r >> 1) + 2 * i + (r & 1)) * 32 + c * 8, vw[i]);

        float s[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[i][e] = 0.f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            uint32_t gs[4], gz[4];
            load_words<16>(rec + P::kGridOff + ((D / 4) * c + 8 * j) * 2, gs);
            load_words<16>(rec + P::kGridOff + P::kGridHalf + ((D / 4) * c + 8 * j) * 2, gz);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t x[4], y[4];
                packed_octet(kw[2 * i][j], gs, gz, x);
                packed_octet(kw[2 * i + 1][j], gs, gz, y);
                const uint32_t f0[4] = {x[0], y[0], x[1], y[1]}, f1[4] = {x[2], y[2], x[3], y[3]};
                tc::mma_16816(s[i], f0, qf[j][0], qf[j][1]);
                tc::mma_16816(s[i], f1, qf[j][2], qf[j][3]);
            }
        }
        uint32_t pt[8];
        softmax(s, pt);
        // the grid of tokens 16 c .. + 16 and this lane's channels (rows r of every tile
        // lie in 64-channel group r / 4 when D = 128)
        uint32_t gs[8], gz[8];
        const uint8_t *grid = vrec + P::kGridOff + (D == 128 ? (r >> 2) * 2 * CHK : 0) + 32 * c;
        load_words<32>(grid, gs);
        load_words<32>(grid + P::kGridHalf, gz);
#pragma unroll
        for (int i = 0; i < NU / 2; ++i) {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const uint32_t s4[4] = {gs[4 * w], gs[4 * w + 1], gs[4 * w + 2], gs[4 * w + 3]};
                const uint32_t z4[4] = {gz[4 * w], gz[4 * w + 1], gz[4 * w + 2], gz[4 * w + 3]};
                uint32_t x[4], y[4];
                packed_octet(vw[2 * i][w], s4, z4, x);
                packed_octet(vw[2 * i + 1][w], s4, z4, y);
                const uint32_t f0[4] = {x[0], y[0], x[1], y[1]}, f1[4] = {x[2], y[2], x[3], y[3]};
                tc::mma_16816(o[i], f0, pt[4 * w], pt[4 * w + 1]);
                tc::mma_16816(o[i], f1, pt[4 * w + 2], pt[4 * w + 3]);
            }
        }
    }

    for (; u < n_units; u += step) {  // window pieces of 16 tokens; rows past n_local read as zeros
        const int t0 = (u - nr) * kPiece;
        const int left = a.n_local - t0;
        const long long row0 = (long long)bg * a.local_stride + t0;
        const uint8_t *kp = reinterpret_cast<const uint8_t *>(a.kl + row0 * D);
        const uint8_t *vp = reinterpret_cast<const uint8_t *>(a.vl + row0 * D);
        uint32_t kx[2][NJ][4], vx[2][NJ][4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int row = 8 * t + r;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                if (row < left) {
                    load_words<16>(kp + (row * D + (D / 4) * c + 8 * j) * 2, kx[t][j]);
                    load_words<16>(vp + (row * D + (D / 4) * c + 8 * j) * 2, vx[t][j]);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) kx[t][j][e] = vx[t][j][e] = 0u;
                }
            }
        }
        float s[1][4] = {{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const uint32_t f0[4] = {kx[0][j][0], kx[1][j][0], kx[0][j][1], kx[1][j][1]};
            const uint32_t f1[4] = {kx[0][j][2], kx[1][j][2], kx[0][j][3], kx[1][j][3]};
            tc::mma_16816(s[0], f0, qf[j][0], qf[j][1]);
            tc::mma_16816(s[0], f1, qf[j][2], qf[j][3]);
        }
        if (r >= left) s[0][0] = s[0][1] = -INFINITY;
        if (8 + r >= left) s[0][2] = s[0][3] = -INFINITY;
        uint32_t pt[2];
        softmax(s, pt);
#pragma unroll
        for (int i = 0; i < NU / 2; ++i) {
            const int j = i >> 1, e = 2 * (i & 1);  // channel tiles 2i, 2i + 1 are pairs e, e + 1 of octet j
            const uint32_t f[4] = {transpose8(vx[0][j][e]), transpose8(vx[0][j][e + 1]), transpose8(vx[1][j][e]),
                                   transpose8(vx[1][j][e + 1])};
            tc::mma_16816(o[i], f, pt[0], pt[1]);
        }
    }

    // this warp's maximum, sum and output
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l_run[h] += __shfl_xor_sync(0xffffffffu, l_run[h], d);
        if (r == 0) {
            wm[warp][2 * c + h] = m_run[h];
            wl[warp][2 * c + h] = l_run[h];
        }
#pragma unroll
        for (int i = 0; i < NU / 2; ++i) {
            const int ch = (D / 4) * (r >> 1) + 4 * i + (r & 1);
            wo[warp][2 * c + h][ch] = o[i][h];
            wo[warp][2 * c + h][ch + 2] = o[i][2 + h];
        }
    }
    __syncthreads();
    // the CTA's: a warp without units has m = -inf and adds nothing
    for (int e = tid; e < G * D; e += kThreads) {
        const int h = e / D, d = e % D;
        float m = wm[0][h];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) m = fmaxf(m, wm[w][h]);
        const float m_sub = m == -INFINITY ? 0.f : m;
        float l = 0.f, acc = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = exp2f(wm[w][h] - m_sub);
            l = fmaf(wl[w][h], f, l);
            acc = fmaf(wo[w][h][d], f, acc);
        }
        if (a.n_cluster == 1) {
            const long long row = (long long)b * a.n_q_heads + (long long)g * G + h;
            a.out[row * D + d] = __float2bfloat16_rn(acc / l);
            if (d == 0) a.lse[row] = (m + log2f(l)) * 0.69314718055994530942f;
        } else {
            co[h][d] = acc;
            if (d == 0) {
                cm[h] = m;
                cl[h] = l;
            }
        }
    }
    if (a.n_cluster == 1) return;
    tc::cluster_arrive();
    tc::cluster_wait();
    // the cluster's: element e of the G x D outputs by CTA rank (e / kThreads) % n_cluster
    const uint32_t sm = tc::smem_u32(cm), sl = tc::smem_u32(cl), so = tc::smem_u32(co);
    for (int e = rank * kThreads + tid; e < G * D; e += a.n_cluster * kThreads) {
        const int h = e / D, d = e % D;
        float mv[kMaxCluster], m = -INFINITY;
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k) {
            mv[k] = k < a.n_cluster ? tc::ld_dsmem_f32(tc::mapa_shared(sm + 4 * h, k)) : -INFINITY;
            m = fmaxf(m, mv[k]);
        }
        const float m_sub = m == -INFINITY ? 0.f : m;
        float l = 0.f, acc = 0.f;
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k)
            if (k < a.n_cluster) {
                const float f = exp2f(mv[k] - m_sub);
                l = fmaf(tc::ld_dsmem_f32(tc::mapa_shared(sl + 4 * h, k)), f, l);
                acc = fmaf(tc::ld_dsmem_f32(tc::mapa_shared(so + 4 * (h * D + d), k)), f, acc);
            }
        const long long row = (long long)b * a.n_q_heads + (long long)g * G + h;
        a.out[row * D + d] = __float2bfloat16_rn(acc / l);
        if (d == 0) a.lse[row] = (m + log2f(l)) * 0.69314718055994530942f;
    }
    // no CTA leaves while another may read its shared memory
    tc::cluster_arrive();
    tc::cluster_wait();
}

// CTAs per (batch, KV head): one wave of the device, at most a unit per warp.
int cluster_size(const hga_params_t &p, int n_local) {
    const int units = (p.topk < p.n_hist_chunks ? p.topk : p.n_hist_chunks) + (n_local + kPiece - 1) / kPiece;
    const long long bg = (long long)p.batch * p.n_kv_heads;
    long long n = (long long)kCtasPerSm * sm_count() / bg;
    const long long most = (units + kWarps - 1) / kWarps;
    if (n > most) n = most;
    if (n > kMaxCluster) n = kMaxCluster;
    return n < 1 ? 1 : (int)n;
}

template <int D> hga_status_t launch_d(const PackedDecodeArgs &a, unsigned bg, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(bg * a.n_cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = a.n_cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, decode_packed_kernel<D>, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    return record_cuda(e);
}

}  // namespace

hga_status_t launch_decode_packed(const hga_params_t &p, const void *q, const uint8_t *hist, int cap, const void *kl,
                                  const void *vl, int n_local, const int32_t *idx, void *out, float *lse,
                                  unsigned *status, cudaStream_t stream) {
    PackedDecodeArgs a;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.hist = hist;
    a.kl = static_cast<const __nv_bfloat16 *>(kl);
    a.vl = static_cast<const __nv_bfloat16 *>(vl);
    a.idx = idx;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse;
    a.status = status;
    a.cap = cap;
    a.local_stride = p.seg_head_stride;
    a.n_q_heads = p.n_q_heads;
    a.n_kv_heads = p.n_kv_heads;
    a.topk = p.topk;
    a.n_hist_chunks = p.n_hist_chunks;
    a.n_local = n_local;
    a.n_cluster = cluster_size(p, n_local);
    a.scale_log2 = (float)(1.4426950408889634 / __builtin_sqrt((double)p.head_dim));
    const unsigned bg = (unsigned)(p.batch * p.n_kv_heads);
    return p.head_dim == 128 ? launch_d<128>(a, bg, stream) : launch_d<64>(a, bg, stream);
}

}  // namespace hga
