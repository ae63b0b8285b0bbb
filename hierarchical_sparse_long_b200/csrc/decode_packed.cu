// Single-query decode over a packed history: one new token per sequence attends, with
// exact softmax, the tokens of its routed 4-bit chunks and its bf16 local window.
//
// "Long-Context Fine-Tuning with Limited VRAM", technical summary section 2.1 (routed
// exact chunks next to a local window), with the history's values as packed.cuh defines
// them: z_t = q . k_t / sqrt(D), out = sum_t softmax(z)_t v_t.
//
// The floor is HBM, and at small batches latency: a routed chunk is 72 D bytes (0.28 of
// bf16), read once for the G <= 8 query heads of its KV head.  A warp takes a whole chunk.
// Its record comes as one bulk copy into the warp's own two-stage ring in shared memory, so
// the next record is on its way while this one is multiplied, and no register holds data in
// flight.  From there the codes are widened straight into MMA operands: the axes that the
// products contract or run along are permuted so that a lane's 16 (K) or 8 (V) bytes of a
// row are exactly its operand registers.  With lane = 4 r + c (r = lane / 4, c = lane % 4):
//   S^T = K Q^T   M = 16 tokens, N = 8 heads.  Row r of token tile t is token
//                 16 (r / 2) + 2 t + r % 2; lane c holds channels c D/4 .. + D/4, which
//                 the k index runs through two pairs at a time (the queries likewise).
//   O^T += V^T P^T  M = 16 channels, N = 8 heads.  Row r of channel tile u is channel
//                 (D/4) (r / 2) + 2 u + r % 2; lane c holds tokens 16 c .. + 16.  P, as
//                 S^T leaves it (tokens by heads), becomes that operand by one
//                 transposing move per 8 tokens.
// The tokens of the window go through the same ring and products in pieces of 16, as bf16.
//
// The units (routed chunks, then window pieces) of one (batch, KV head) are dealt to the
// warps of a thread-block cluster; every warp keeps its own running maximum, sum and
// output, which are merged through shared memory, first of the CTA, then of the
// cluster: one launch, no workspace, sums in a fixed order.
//
// Measured: 13.8 us for 16 sequences of 32 + 8 heads at 32 routed chunks and 64 window tokens
// (42 MB, 3.1 TB/s of the 6.5 that a copy reaches), 4.9 us for one at 16 chunks.  No pipe is
// full there (issue slots 38%, integer pipe 34%, DRAM 30% of their peaks): a unit is a chain of
// about 1,040 instructions of one warp (1.2 us, 1.9 with two CTAs on the SM), and with 256 CTAs on
// 148 SMs, some holding one and some two, a scheduler has 1.7 warps to choose from; 36 units over 8
// warps are five rounds of them.  The rest is the start (routes, then first records) and the
// merge.  With loads into registers in place of the ring, and a merge by CTA and then by
// cluster, the 16 sequences took 19.6 us.
#include <cstddef>

#include "dependent.cuh"
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
constexpr int kCtasPerSm = 3;   // at most 168 registers a thread; 72 KiB of rings a CTA
constexpr unsigned kSmBytes = 228 * 1024;  // shared memory of an SM
constexpr int kStages = 2;      // one unit multiplied, one on its way

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
    int merge_groups, merge_shift;  // groups of four outputs per CTA, log2 of the lanes of one
    float scale_log2;  // log2(e) / sqrt(D)
};

// Transposes the 8x8 b16 matrix of which lane 4 r + c holds (row r, columns 2 c, 2 c + 1).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// N bytes (a multiple of 8) of a ring stage.
template <int N> __device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&w)[N / 4]) {
#pragma unroll
    for (int i = 0; i < N / 16; ++i) {
        const uint4 v = *(reinterpret_cast<const uint4 *>(p) + i);
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
    }
    if constexpr (N % 16 == 8) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p + N / 16 * 16);
        w[N / 4 - 2] = v.x;
        w[N / 4 - 1] = v.y;
    }
}

// 16 bytes of shared memory of the cluster.
__device__ __forceinline__ float4 load_peer(uint32_t addr) {
    const uint4 v = tc::ld_dsmem_v4(addr);
    return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}

// Partial results of a CTA's warps: maximum and sum by head, outputs in quarters of a row
// with pads that spread a warp's stores over the banks.
template <int D> struct Merge {
    static constexpr int kQuarter = D / 4 + 4, kRow = 4 * kQuarter + 4;
    float4 m[kHeads], l[kHeads];  // of the four warps
    float o[kWarps][kHeads][kRow];
};
static_assert(kWarps == 4, "a head's maxima of a CTA are one float4");

template <int D>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) decode_packed_kernel(const PackedDecodeArgs a) {
    using P = Packed<D>;
    constexpr int NJ = D / 32;  // channel octets of a lane
    constexpr int NU = D / 8;   // 8-channel row tiles
    static_assert(4 * kPiece * D <= P::kRecord, "a window piece fits a ring stage");
    using M = Merge<D>;
    static_assert(sizeof(M) <= kWarps * kStages * P::kRecord, "the merge reuses the rings");
    extern __shared__ __align__(16) uint8_t rings[];  // [kWarps][kStages][record]
    __shared__ int units[kWarps][kMaxRouted];
    __shared__ uint64_t full[kWarps][kStages];
    __shared__ int abort_flag;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = lane >> 2, c = lane & 3;
    const int G = a.n_q_heads / a.n_kv_heads;
    const int rank = (int)blockIdx.x % a.n_cluster;
    const int bg = (int)blockIdx.x / a.n_cluster;
    const int b = bg / a.n_kv_heads, g = bg % a.n_kv_heads;

    depend_wait();
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
    if (tid == 0) abort_flag = 0;
    if (lane == 0) {
        for (int s = 0; s < kStages; ++s) tc::mbar_init(&full[warp][s], 1);
        tc::fence_mbar_init();
    }
    int nr = 0;
    {  // the valid routes, in order; -1 is padding, anything else out of range is skipped
        const int32_t *sel = a.idx + (long long)bg * a.topk;
#pragma unroll
        for (int i0 = 0; i0 < kMaxRouted; i0 += 32) {
            const int j = i0 + lane < a.topk ? sel[i0 + lane] : -1;
            const bool ok = j >= 0 && j < a.n_hist_chunks;
            if (!ok && j != -1 && rank == 0 && warp == 0) atomicOr(a.status, kDevBadIndex);
            const unsigned m = __ballot_sync(0xffffffffu, ok);
            if (ok) units[warp][nr + __popc(m & ((1u << lane) - 1u))] = j;
            nr += __popc(m);
        }
    }
    __syncwarp();
    const int n_units = nr + (a.n_local + kPiece - 1) / kPiece;
    const int step = a.n_cluster * kWarps;
    // a warp's units interleave over the CTAs first, so that few units use every SM
    const int u0 = warp * a.n_cluster + rank;
    uint8_t *ring = rings + warp * kStages * P::kRecord;
    // unit u into stage s: a record, or a window piece's K rows and V rows
    auto fetch = [&](int u, int s) {
        if (lane != 0) return;
        uint8_t *dst = ring + s * P::kRecord;
        if (u < nr) {
            tc::mbar_arrive_expect_tx(&full[warp][s], P::kRecord);
            tc::bulk_load(dst, a.hist + ((long long)bg * a.cap + units[warp][u]) * P::kRecord, P::kRecord,
                          &full[warp][s]);
        } else {
            const int t0 = (u - nr) * kPiece;
            const int n = a.n_local - t0 < kPiece ? a.n_local - t0 : kPiece;
            const long long row0 = (long long)bg * a.local_stride + t0;
            tc::mbar_arrive_expect_tx(&full[warp][s], 4 * n * D);
            tc::bulk_load(dst, a.kl + row0 * D, 2 * n * D, &full[warp][s]);
            tc::bulk_load(dst + 2 * kPiece * D, a.vl + row0 * D, 2 * n * D, &full[warp][s]);
        }
    };
    if (u0 < n_units) fetch(u0, 0);

    // state of heads 2c, 2c + 1: o[i] rows r (channel tile 2i) and r + 8 (tile 2i + 1)
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};  // l: this lane's tokens only
    float o[NU / 2][4];
#pragma unroll
    for (int i = 0; i < NU / 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    __syncthreads();  // abort_flag

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
        // P is rounded to bf16 for the product, as in the other attention kernels: the tensor
        // cores' bf16 products take no wider P, and the row sum is of the unrounded one.  Outputs
        // are 2.1e-3 in norm off those of 64 bits, 1.7e-3 with P in fp32 (their own rounding).
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            pt[2 * i] = transpose8(tc::pack_bf16(s[i][0], s[i][1]));
            pt[2 * i + 1] = transpose8(tc::pack_bf16(s[i][2], s[i][3]));
        }
    };

    auto chunk = [&](const uint8_t *rec) {
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
    };

    // a window piece of 16 tokens, `left` of them in the window: rows past that read as zeros
    auto piece = [&](const uint8_t *kp, int left) {
        const uint8_t *vp = kp + 2 * kPiece * D;
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
    };

    bool ok = true;
    for (int u = u0, i = 0; ok && u < n_units; u += step, ++i) {
        uint64_t *bar = &full[warp][i & 1];
        ok = __all_sync(0xffffffffu, tc::mbar_wait(bar, (i >> 1) & 1, &abort_flag, a.status));
        if (!ok) {  // the copy still lands before the ring is used again
            int never = 0;
            tc::mbar_wait(bar, (i >> 1) & 1, &never, a.status, 1ll << 28);
            break;
        }
        // the next unit, into the stage that the previous one left: not before this one has
        // arrived, so that the first units of all warps share the bandwidth of the start
        if (u + step < n_units) fetch(u + step, (i + 1) & 1);
        const uint8_t *rec = ring + (i & 1) * P::kRecord;
        if (u < nr) {
            chunk(rec);
        } else {
            piece(rec, a.n_local - (u - nr) * kPiece);
        }
        __syncwarp();  // every lane has read the stage
    }
    depend_next();
    __syncthreads();  // the rings are free

    // this warp's maximum, sum and output
    M &mg = *reinterpret_cast<M *>(rings);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l_run[h] += __shfl_xor_sync(0xffffffffu, l_run[h], d);
        if (r == 0) {
            reinterpret_cast<float *>(&mg.m[2 * c + h])[warp] = m_run[h];
            reinterpret_cast<float *>(&mg.l[2 * c + h])[warp] = l_run[h];
        }
        float *row = &mg.o[warp][2 * c + h][M::kQuarter * (r >> 1) + (r & 1)];
#pragma unroll
        for (int i = 0; i < NU / 2; ++i) {
            row[4 * i] = o[i][h];
            row[4 * i + 2] = o[i][2 + h];
        }
    }
    // The sum over all warps of the cluster, in a fixed order.  Four outputs belong to kl
    // lanes, one for each CTA (a power of two of them), which reads that CTA's four warps;
    // the lanes' sums then meet in shuffles.  The groups of four are dealt evenly to the CTAs.
    // A warp without units, and a lane past the cluster's end, has m = -inf and adds nothing.
    const int nc = a.n_cluster, kl = 1 << a.merge_shift;
    if (nc > 1) tc::cluster_arrive();
    const int end = min((rank + 1) * a.merge_groups, G * D / 4);
    const int k = tid & (kl - 1);
    int e0 = rank * a.merge_groups;
    if (nc > 1)
        tc::cluster_wait();
    else
        __syncthreads();
#pragma unroll 1
    for (; e0 < end; e0 += kThreads >> a.merge_shift) {
        const int e = min(e0 + (tid >> a.merge_shift), end - 1);
        const int h = e / (D / 4), d4 = e % (D / 4);
        float4 mv = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY), lv = make_float4(0.f, 0.f, 0.f, 0.f);
        float4 ov[kWarps] = {lv, lv, lv, lv};
        if (k < nc) {
            const uint32_t sm = tc::mapa_shared(tc::smem_u32(&mg), k);
            mv = load_peer(sm + (uint32_t)offsetof(M, m) + 16 * h);
            lv = load_peer(sm + (uint32_t)offsetof(M, l) + 16 * h);
            const uint32_t at = 4 * (h * M::kRow + M::kQuarter * (d4 / (D / 16)) + 4 * (d4 % (D / 16)));
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                ov[w] = load_peer(sm + (uint32_t)offsetof(M, o) + w * (uint32_t)sizeof(mg.o[0]) + at);
        }
        float m = fmaxf(fmaxf(mv.x, mv.y), fmaxf(mv.z, mv.w));
#pragma unroll 1
        for (int o = kl / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float m_sub = m == -INFINITY ? 0.f : m;
        const float f[4] = {tc::ex2(mv.x - m_sub), tc::ex2(mv.y - m_sub), tc::ex2(mv.z - m_sub), tc::ex2(mv.w - m_sub)};
        float v[5] = {lv.x * f[0] + lv.y * f[1] + lv.z * f[2] + lv.w * f[3], 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            v[1] = fmaf(ov[w].x, f[w], v[1]);
            v[2] = fmaf(ov[w].y, f[w], v[2]);
            v[3] = fmaf(ov[w].z, f[w], v[3]);
            v[4] = fmaf(ov[w].w, f[w], v[4]);
        }
#pragma unroll 1
        for (int o = kl / 2; o; o >>= 1)
#pragma unroll
            for (int i = 0; i < 5; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        if (k == 0 && e0 + (tid >> a.merge_shift) < end) {
            const long long row = (long long)b * a.n_q_heads + (long long)g * G + h;
            const float inv = 1.f / v[0];
            *reinterpret_cast<uint2 *>(a.out + row * D + 4 * d4) =
                make_uint2(tc::pack_bf16(v[1] * inv, v[2] * inv), tc::pack_bf16(v[3] * inv, v[4] * inv));
            if (d4 == 0) a.lse[row] = (m + log2f(v[0])) * 0.69314718055994530942f;
        }
    }
    if (nc == 1) return;
    // no CTA leaves while another may read its shared memory
    tc::cluster_arrive();
    tc::cluster_wait();
}

// CTAs per (batch, KV head): 1, 2, 4 or 8 (clusters of three took longer than their work
// predicts), all resident at once.  With c CTAs on an SM a warp takes about 0.4 + 0.8 c us
// per unit of D = 128 (1.16 alone, 1.87, 2.75 measured), and a cluster's merge about 0.5 us,
// 1 us for eight CTAs; the least sum of both is taken.  Measured, us for 1 / 2 / 4 / 8 CTAs:
//   8 pairs of 19 units    8.1 /  6.3 /  5.1 /  5.0      32 pairs of 19   8.2 /  6.3 /  5.7 /  6.6
//   128 pairs of 36       14.7 / 13.8 / 20.0 / 26.8     192 pairs of 36  20.9 / 17.8 / 23.7 / 37.0
// D = 64, whose units are half as long, keeps the order:
//   8 pairs of 20 units    6.1 /  5.1 /  4.3 /  4.3      32 pairs of 36   9.8 /  6.9 /  5.7 /  6.4
//   96 pairs of 49        13.2 / 11.1 /  9.7 / 15.9     192 pairs of 49  17.6 / 14.6 / 20.2 / 27.5
int cluster_size(const hga_params_t &p, int n_local) {
    const long long units =
        (p.topk < p.n_hist_chunks ? p.topk : p.n_hist_chunks) + ((long long)n_local + kPiece - 1) / kPiece;
    const long long bg = (long long)p.batch * p.n_kv_heads, sms = sm_count();
    int best = 1;
    long long best_cost = 0;
    for (int n = 1; n <= kMaxCluster && (n == 1 || bg * n <= kCtasPerSm * sms); n *= 2) {
        const long long serial = (units + kWarps * n - 1) / (kWarps * n), on_sm = (bg * n + sms - 1) / sms;
        const long long cost = serial * (4 + 8 * on_sm) + (n == 1 ? 0 : n == 8 ? 10 : 5);  // tenths of a us
        if (n == 1 || cost < best_cost) {
            best = n;
            best_cost = cost;
        }
    }
    return best;
}

template <int D> hga_status_t launch_d(const PackedDecodeArgs &a, unsigned bg, cudaStream_t stream) {
    // The CTAs come to SMs that the previous kernel leaves one after another; with room for
    // more of them than their even share, the first SMs take too many (16.1 against 14.3 us
    // per call of 256 CTAs in a graph).  So each asks for more than a (share + 1)-th of the
    // shared memory.
    const unsigned grid = bg * a.n_cluster, sms = (unsigned)sm_count(), share = (grid + sms - 1) / sms;
    int smem = kWarps * kStages * Packed<D>::kRecord;
    if (share <= kCtasPerSm && smem < (int)(kSmBytes / (share + 1))) smem = (int)(kSmBytes / (share + 1));
    const cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void *>(decode_packed_kernel<D>), smem);
    if (e != cudaSuccess) return record_cuda(e);
    return record_cuda(launch_dependent(decode_packed_kernel<D>, grid, kThreads, smem, a.n_cluster, stream, a));
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
    a.merge_groups = (p.n_q_heads / p.n_kv_heads * p.head_dim / 4 + a.n_cluster - 1) / a.n_cluster;
    a.merge_shift = a.n_cluster == 1 ? 0 : a.n_cluster == 2 ? 1 : a.n_cluster <= 4 ? 2 : 3;
    a.scale_log2 = (float)(1.4426950408889634 / __builtin_sqrt((double)p.head_dim));
    const unsigned bg = (unsigned)(p.batch * p.n_kv_heads);
    return p.head_dim == 128 ? launch_d<128>(a, bg, stream) : launch_d<64>(a, bg, stream);
}

}  // namespace hga
