// Exact-token attention forward over a packed history on the 5th-generation tensor cores
// (tcgen05 / TMEM / TMA): bf16 queries and segment, 4-bit history (packed.cuh), fp32
// accumulation, head_dim 64 or 128.
//
// "Long-Context Fine-Tuning with Limited VRAM", technical summary section 2.1 (exact K/V
// of the routed chunks attended with a local window): what attn_fwd_tc.cu computes, with
// the history's keys and values read as the values of their 4-bit records.
//
// One CTA per (batch, kv head, query block, head sub-group), as in attn_fwd_tc.cu: HC = 4,
// 2 or 1 query heads of a KV group as NH M=128 halves share every 64-token tile.  The
// records are widened inside the kernel, on four warps beside the ones that run the
// softmax, so no bf16 copy of the history exists anywhere and a routed chunk costs 9 KiB
// of HBM / L2 reads instead of 32.
//
// Warp roles (NH = 2: 512 threads):
//   warps 0, 2  QK issuers of halves 0, 1 (warp 0 also owns TMEM):
//               S_h = Q_h K^T  (M128 N64 KD, K-major A and B, SW128)
//   warps 1, 3  PV issuers: O_h += P_h V  (M128 ND K64, P from TMEM)
//   then 4 NH   softmax warps: one TMEM lane (= query row) per thread, online softmax in
//               the log2 domain, P written back as bf16 pairs into the tile's S buffer
//   last 4      producers.  History tiles: records come as bulk copies into a ring of
//               three in shared memory; a thread reads its share of the codes and grids,
//               widens it and stores 16 bytes per word into the K / V stage: K as
//               [D / 64][64 tokens][128 B of channels], V transposed as [D channels][128 B
//               of tokens] -- the record's own order, so one word is one swizzled 16-byte
//               chunk in both -- hence V is K-major for these tiles.  Segment tiles: TMA, V
//               as rows of tokens (MN-major); the PV issuers pick descriptor and instruction
//               by tile.
// A K (V) stage is full when all four producer warps have arrived; for a segment tile one
// of them arrives with the byte count of its TMA boxes.
// TMEM (512 columns): O_h at 128h, S_h double-buffered at 256 + 128h + 64b.
// Every wait is bounded; a timeout sets HGA_DEV_TIMEOUT and the CTA unwinds.
//
// Measured: 74.1 us for the last 2,048 queries of 16K (32 + 8 heads, 68.7 GFLOP: 927
// TFLOP/s), 254 us for the last 4,096 of 128K (275 GFLOP: 1,083 TFLOP/s), in bursts; for
// seconds on end the power cap makes them 80.5 and 291 us.  A 64-token tile of
// two halves takes about 1,950 cycles, of which its products' operand traffic from shared
// memory accounts for about 1,470 (a QK product re-reads its 128 rows of queries for 64
// keys); a half's softmax (about 1,500) and products overlap with the other half's.  D = 64 takes
// 66.5 us for the 16K segment (34 GFLOP: 517 TFLOP/s): half the products for the same softmax.
// Groups that are no multiple of 4 run on one half, an odd head with 64 of its 128 rows spare:
// 162.6 us for 24 + 8 heads of 128, 187.6 for 28 + 4 (317 and 321 TFLOP/s).  128-token
// tiles, which re-read the queries half as often, left room for one score buffer per half and
// took 2,300 cycles per 64 tokens: softmax and products of a half no longer overlap.
#include "dependent.cuh"
#include "packed.cuh"
#include "tc_issue.cuh"
#include "tc_ptx.cuh"

namespace hga {

namespace {

constexpr int TILE = 64;
constexpr int NSTAGE = 4;
constexpr float kRescaleLog2 = 8.f;  // lazy-rescale threshold on the running max (log2 units)
constexpr int kIssueWarps = 4;
constexpr int kProdWarps = 4;
constexpr int kRecStages = 3;  // records on their way to, or in, shared memory

template <int D, int NH> struct Smem {
    static constexpr uint32_t Q_HALF = 128 * D * 2;   // [D / 64][128 rows][128 B]
    static constexpr uint32_t KV_TILE = TILE * D * 2;  // K [D / 64][64 rows][128 B]; V also [D rows][128 B]
    static constexpr uint32_t Q = 0;
    static constexpr uint32_t K = Q + NH * Q_HALF;
    static constexpr uint32_t V = K + NSTAGE * KV_TILE;
    static constexpr uint32_t REC = V + NSTAGE * KV_TILE;  // [kRecStages][record]
    static constexpr uint32_t BAR = (REC + kRecStages * Packed<D>::kRecord + 1023) / 1024 * 1024;
    static constexpr uint32_t TOTAL = BAR + 1024;
    static constexpr uint32_t ALLOC = TOTAL + 1024;  // + alignment slack
};

// D[tmem] (+)= A[tmem] * B[smem] for one K=16 step of kind::f16 (A read from TMEM).
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 2D tiled store of shared memory (visible to the async proxy) to (x, y), in this thread's
// bulk group; the wait returns once the group's stores are done.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, const void *src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(tc::smem_u32(src))
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

struct Bars {
    uint64_t q_full;
    uint64_t k_full[NSTAGE];
    uint64_t k_empty[NSTAGE];  // released once QK^T of the tile completes (both halves)
    uint64_t v_full[NSTAGE];
    uint64_t v_empty[NSTAGE];  // released once PV of the tile completes (both halves)
    uint64_t r_full[kRecStages];   // a record in shared memory
    uint64_t r_empty[kRecStages];  // and read by the producer warps
    uint64_t s_full[2][2];     // [half][S/P buffer]: S of the buffer's tile in TMEM
    uint64_t p_full[2][2];     // [half][S/P buffer]: P of the buffer's tile written to TMEM
    uint64_t o_done[2][2];     // [half][S/P buffer]: PV of the buffer's tile completed
    uint64_t drain[4];         // one per issuing warp (abort path)
    uint32_t tmem_base;
    int abort;
    int n_hist;
    int sm0_tiles;  // tiles whose softmax half 0 has finished (scheduling hint)
    int tiles[64];
};
static_assert(sizeof(Bars) <= 1024, "barrier block must fit its region");

struct FwdPackedArgs {
    int batch, n_q_heads, n_kv_heads, seg_len, topk, n_hist_chunks;
    int n_sub, hc;  // CTAs per KV group, query heads per CTA (4, 2 or 1)
    long long seg_stride, cap;
    int qb0, n_blocks, n_first;
    const uint8_t *hist;
    const int32_t *idx;
    float *lse;
    unsigned *status;
    float scale_log2;  // log2(e) / sqrt(D)
};

// Bounded wait until the shared counter reaches `target` (same contract as mbar_wait).
__device__ __forceinline__ bool wait_count(int *counter, int target, volatile int *abort, unsigned *status) {
    volatile int *c = counter;
    if (*c >= target) return true;
    const long long t0 = clock64();
    while (*c < target) {
        if (*abort) return false;
        if (clock64() - t0 > (1ll << 31)) {
            *abort = 1;
            atomicOr(status, kDevTimeout);
            return false;
        }
    }
    return true;
}

// (x0, x1) y + z, and (d0, d1) += (x0, x1): two elements per instruction.
__device__ __forceinline__ void fma2(float &x0, float &x1, float y, float z) {
    asm("{\n\t.reg .b64 a, b, c;\n\t"
        "mov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\tmov.b64 c, {%3, %3};\n\t"
        "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(x0), "+f"(x1)
        : "f"(y), "f"(z));
}
__device__ __forceinline__ void add2(float &d0, float &d1, float x0, float x1) {
    asm("{\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
        "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(d0), "+f"(d1)
        : "f"(x0), "f"(x1));
}

// Codes and grid of one thread's share of a K part: octet `o` of every kStep-th token from r0.
template <int D> struct KShare {
    static constexpr int kOctets = D / 8, kStep = 32 * kProdWarps / kOctets, kWords = TILE / kStep;
    uint32_t w[kWords], s[4], z[4];
    __device__ __forceinline__ void load(const uint8_t *rec, int o, int r0) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const uint32_t *>(rec)[(r0 + kStep * i) * kOctets + o];
        const uint4 a = reinterpret_cast<const uint4 *>(rec + Packed<D>::kGridOff)[o];
        const uint4 b = reinterpret_cast<const uint4 *>(rec + Packed<D>::kGridOff + Packed<D>::kGridHalf)[o];
        s[0] = a.x; s[1] = a.y; s[2] = a.z; s[3] = a.w;
        z[0] = b.x; z[1] = b.y; z[2] = b.z; z[3] = b.w;
    }
};
// The same of a V part: token octet `o` of every 16th channel from r0 (four to a group).
template <int D> struct VShare {
    static constexpr int kWords = D / 16;
    uint32_t w[kWords], s[D / 64][4], z[D / 64][4];
    __device__ __forceinline__ void load(const uint8_t *vrec, int o, int r0) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const uint32_t *>(vrec)[(r0 + 16 * i) * 8 + o];
#pragma unroll
        for (int gp = 0; gp < D / 64; ++gp) {
            const uint8_t *grid = vrec + Packed<D>::kGridOff + gp * 2 * TILE;
            const uint4 a = reinterpret_cast<const uint4 *>(grid)[o];
            const uint4 b = reinterpret_cast<const uint4 *>(grid + Packed<D>::kGridHalf)[o];
            s[gp][0] = a.x; s[gp][1] = a.y; s[gp][2] = a.z; s[gp][3] = a.w;
            z[gp][0] = b.x; z[gp][1] = b.y; z[gp][2] = b.z; z[gp][3] = b.w;
        }
    }
};

template <int D, int NH>
__global__ void __launch_bounds__(32 * (kIssueWarps + 4 * NH + kProdWarps), 1)
    attn_fwd_packed_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_ks,
                           const __grid_constant__ CUtensorMap tm_vs, const __grid_constant__ CUtensorMap tm_o,
                           const FwdPackedArgs a) {
    using L = Smem<D, NH>;
    constexpr uint32_t IDESC_QK = tc::idesc_bf16(128, TILE, false, false);
    constexpr uint32_t IDESC_PV = tc::idesc_bf16(128, D, false, true);        // segment: V rows are tokens
    constexpr uint32_t IDESC_PV_HIST = tc::idesc_bf16(128, D, false, false);  // history: V rows are channels
    constexpr int kSoftmax0 = kIssueWarps, kProd0 = kIssueWarps + 4 * NH;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Bars *bars = reinterpret_cast<Bars *>(smem + L::BAR);
    const uint32_t sbase = tc::smem_u32(smem);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nqb = a.seg_len / TILE;
    const int n_units = a.batch * a.n_kv_heads * a.n_sub;
    // longest (latest) blocks first, behind `n_first` of the shortest
    const int n_ctas = (int)gridDim.x, x = (int)blockIdx.x;
    const int order = x < a.n_first ? n_ctas - a.n_first + x : x - a.n_first;
    const int m = a.qb0 + a.n_blocks - 1 - order / n_units;
    const int unit = order % n_units;
    const int bg = unit / a.n_sub;
    const int b = bg / a.n_kv_heads, g = bg % a.n_kv_heads;
    // first query head of this CTA: the KV group's heads g*G .., HC per CTA
    const int h0 = g * (a.n_q_heads / a.n_kv_heads) + (unit % a.n_sub) * a.hc;

    if (threadIdx.x == 0) {
        tc::mbar_init(&bars->q_full, 1);
        for (int s = 0; s < NSTAGE; ++s) {
            tc::mbar_init(&bars->k_full[s], kProdWarps);
            tc::mbar_init(&bars->k_empty[s], NH);
            tc::mbar_init(&bars->v_full[s], kProdWarps);
            tc::mbar_init(&bars->v_empty[s], NH);
        }
        for (int s = 0; s < kRecStages; ++s) {
            tc::mbar_init(&bars->r_full[s], 1);
            tc::mbar_init(&bars->r_empty[s], kProdWarps);
        }
        for (int h = 0; h < 2; ++h)
            for (int bb = 0; bb < 2; ++bb) {
                tc::mbar_init(&bars->s_full[h][bb], 1);
                tc::mbar_init(&bars->p_full[h][bb], 4);  // every softmax warp of the half
                tc::mbar_init(&bars->o_done[h][bb], 1);
            }
        for (int d = 0; d < 4; ++d) tc::mbar_init(&bars->drain[d], 1);
        bars->sm0_tiles = 0;
        bars->abort = 0;
        tc::fence_mbar_init();
    }
    if (warp == 0) tc::tmem_alloc<512>(&bars->tmem_base);
    depend_wait();
    if (warp == 1) {  // the block's valid routes, in order; -1 is padding, anything else is skipped and flagged
        const int32_t *sel = a.idx + ((long long)bg * nqb + m) * a.topk;
        int n = 0;
#pragma unroll
        for (int i0 = 0; i0 < 64; i0 += 32) {
            const int j = i0 + lane < a.topk ? sel[i0 + lane] : -1;
            const bool ok = j >= 0 && j < a.n_hist_chunks;
            if (!ok && j != -1) atomicOr(a.status, kDevBadIndex);
            const unsigned mask = __ballot_sync(0xffffffffu, ok);
            if (ok) bars->tiles[n + __popc(mask & ((1u << lane) - 1u))] = j;
            n += __popc(mask);
        }
        if (lane == 0) bars->n_hist = n;
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = bars->tmem_base;
    volatile int *abort = &bars->abort;
    const int n_hist = bars->n_hist;          // history tiles, then segment tiles 0 .. m
    const int n_tiles = n_hist + m + 1;
    int issued = 0;   // producer warp 0: tiles whose loads it has issued, and
    int records = 0;  // records asked for (drained on abort)

    if (warp < kIssueWarps) {
        // ------------------------------------------------------------ UMMA issuers
        const int h = warp >> 1;           // M half
        const bool qk = (warp & 1) == 0;   // warps 0, 2: QK^T; warps 1, 3: PV
        if (h < NH) {
            // The whole warp runs the loop (waits included) and elects one lane per MMA.
            // Descriptors are built once; a K-step, stage or buffer offset is added
            // to the start-address field (addresses stay below 2^18, so no carry).
            bool ok = true;
            if (qk) {
                const uint64_t q_desc = tc::desc_sw128(sbase + L::Q + h * L::Q_HALF, 16, 1024);
                const uint64_t k_desc = tc::desc_sw128(sbase + L::K, 16, 1024);
                ok = __all_sync(0xffffffffu, tc::mbar_wait(&bars->q_full, 0, abort, a.status));
                for (int j = 0; ok && j < n_tiles; ++j) {
                    const int s = j % NSTAGE, bb = j & 1;
                    if (!__all_sync(0xffffffffu, tc::mbar_wait(&bars->k_full[s], (j / NSTAGE) & 1, abort, a.status)))
                        break;
                    // S buffer bb is free once PV(j-2), which read P(j-2) from it, has completed
                    if (j >= 2 && !__all_sync(0xffffffffu, tc::mbar_wait(&bars->o_done[h][bb], ((j >> 1) - 1) & 1,
                                                                         abort, a.status)))
                        break;
                    // half 1 runs half a tile behind half 0, so that the two softmax groups
                    // take turns on the MUFU
                    if (h == 1 && j >= 1 && !__all_sync(0xffffffffu, wait_count(&bars->sm0_tiles, j, abort, a.status)))
                        break;
                    tc::fence_after_sync();
                    const uint64_t kd = k_desc + (uint64_t)((s * L::KV_TILE) >> 4);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t koff = ((kk >> 2) * (64 * 128) + (kk & 3) * 32) >> 4;
                        const uint32_t qoff = ((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4;
                        if (tc::elect_one())
                            tc::mma_f16(tmem + 256 + 128 * h + 64 * bb, q_desc + qoff, kd + koff, IDESC_QK,
                                        kk > 0 ? 1u : 0u);
                        __syncwarp();
                    }
                    if (tc::elect_one()) {
                        tc::mma_commit(&bars->s_full[h][bb]);
                        tc::mma_commit(&bars->k_empty[s]);  // one arrival per half
                    }
                    __syncwarp();
                }
            } else {
                const uint64_t v_seg = tc::desc_sw128(sbase + L::V, 8192, 1024);  // rows of tokens
                const uint64_t v_hist = tc::desc_sw128(sbase + L::V, 16, 1024);   // rows of channels
                const uint32_t o_tmem = tmem + 128 * h;
                for (int t = 0; t < n_tiles; ++t) {
                    const int s = t % NSTAGE, pb = t & 1;
                    if (!__all_sync(0xffffffffu, tc::mbar_wait(&bars->v_full[s], (t / NSTAGE) & 1, abort, a.status) &&
                                                     tc::mbar_wait(&bars->p_full[h][pb], (t >> 1) & 1, abort,
                                                                   a.status)))
                        break;
                    tc::fence_after_sync();
                    // P(t) as bf16 pairs in the first 32 columns of S buffer pb: 8 columns per K step.
                    // The instruction descriptors are constants: with a run-time one an issue
                    // takes twice as long.
                    const uint32_t pa = tmem + 256 + 128 * h + 64 * pb;
                    const uint64_t voff = (uint64_t)((s * L::KV_TILE) >> 4);
                    if (t < n_hist) {
#pragma unroll
                        for (int kk = 0; kk < TILE / 16; ++kk) {
                            if (tc::elect_one())
                                mma_f16_ts(o_tmem, pa + 8 * kk, v_hist + voff + (uint64_t)(kk * (32 >> 4)),
                                           IDESC_PV_HIST, (t > 0 || kk > 0) ? 1u : 0u);
                            __syncwarp();
                        }
                    } else {
#pragma unroll
                        for (int kk = 0; kk < TILE / 16; ++kk) {
                            if (tc::elect_one())
                                mma_f16_ts(o_tmem, pa + 8 * kk, v_seg + voff + (uint64_t)(kk * (2048 >> 4)), IDESC_PV,
                                           (t > 0 || kk > 0) ? 1u : 0u);
                            __syncwarp();
                        }
                    }
                    if (tc::elect_one()) {
                        tc::mma_commit(&bars->o_done[h][pb]);
                        tc::mma_commit(&bars->v_empty[s]);  // one arrival per half
                    }
                    __syncwarp();
                }
            }
        }
    } else if (warp >= kProd0) {
        // ------------------------------------------------------------ producers
        const int t = (warp - kProd0) * 32 + lane;
        const int ko = t % KShare<D>::kOctets, kr = t / KShare<D>::kOctets;  // K: channel octet, first token
        const int vo = t & 7, vr = t >> 3;   // V: token octet, first channel
        // swizzle: a row's 16-byte chunk index is XORed with the row index mod 8, which
        // is the same for all rows of a thread
        const uint32_t kdst = sbase + L::K + (ko >> 3) * (64 * 128) + kr * 128 + (((ko & 7) ^ (kr & 7)) << 4);
        const uint32_t vdst = sbase + L::V + vr * 128 + ((vo ^ (vr & 7)) << 4);
        const uint8_t *base = a.hist + (long long)bg * a.cap * Packed<D>::kRecord;
        // the next record, as one bulk copy: ahead by kRecStages tiles, and without loads in
        // flight in the threads, for which a proxy fence would wait
        auto fetch = [&]() {
            uint64_t *bar = &bars->r_full[records % kRecStages];
            tc::mbar_arrive_expect_tx(bar, Packed<D>::kRecord);
            tc::bulk_load(smem + L::REC + (records % kRecStages) * Packed<D>::kRecord,
                          base + (long long)bars->tiles[records] * Packed<D>::kRecord, Packed<D>::kRecord, bar);
            ++records;
        };
        if (t == 0) {
            while (records < n_hist && records < kRecStages) fetch();
            tc::tma_prefetch_desc(&tm_q);
            tc::tma_prefetch_desc(&tm_ks);
            tc::tma_prefetch_desc(&tm_vs);
            tc::mbar_arrive_expect_tx(&bars->q_full, NH * L::Q_HALF);
            for (int hh = 0; hh < 2 * NH; ++hh) {
                const int qrow = (b * a.n_q_heads + h0 + (a.hc == 1 ? 0 : hh)) * a.seg_len + m * TILE;
                uint8_t *dst = smem + L::Q + (hh >> 1) * L::Q_HALF + (hh & 1) * (64 * 128);
                for (int c = 0; c < D / 64; ++c)
                    tc::tma_load_2d(dst + c * (128 * 128), &tm_q, 64 * c, qrow, &bars->q_full);
            }
        }
        __syncwarp();
        // a segment tile, or a warp's arrival for it
        auto seg_tile = [&](uint8_t *dst, const CUtensorMap *map, int j, uint64_t *bar) {
            if (t == 0) {
                const int row = (int)((long long)bg * a.seg_stride + (long long)(j - n_hist) * TILE);
                tc::mbar_arrive_expect_tx(bar, L::KV_TILE);
                for (int c = 0; c < D / 64; ++c) tc::tma_load_2d(dst + c * (64 * 128), map, 64 * c, row, bar);
            } else if (lane == 0) {
                tc::mbar_arrive(bar);
            }
            __syncwarp();
        };
        for (int j = 0; j < n_tiles; ++j) {
            const int s = j % NSTAGE, u = j / NSTAGE;
            // this thread's codes and grids of the tile, out of the record's stage
            KShare<D> ks;
            VShare<D> vs;
            const int rs = j % kRecStages;
            if (j < n_hist) {
                if (!__all_sync(0xffffffffu, tc::mbar_wait(&bars->r_full[rs], (j / kRecStages) & 1, abort, a.status)))
                    break;
                const uint8_t *rec = smem + L::REC + rs * Packed<D>::kRecord;
                ks.load(rec, ko, kr);
                vs.load(rec + Packed<D>::kPart, vo, vr);
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bars->r_empty[rs]);
            }
            // a stage frees once the products of the tile NSTAGE back have read it
            if (j >= NSTAGE &&
                !__all_sync(0xffffffffu, tc::mbar_wait(&bars->k_empty[s], (u - 1) & 1, abort, a.status) &&
                                             tc::mbar_wait(&bars->v_empty[s], (u - 1) & 1, abort, a.status)))
                break;
            if (j < n_hist) {
#pragma unroll
                for (int i = 0; i < KShare<D>::kWords; ++i) {
                    uint32_t r[4];
                    packed_octet(ks.w[i], ks.s, ks.z, r);
                    tc::st_shared_v4(kdst + s * L::KV_TILE + i * KShare<D>::kStep * 128, r[0], r[1], r[2], r[3]);
                }
#pragma unroll
                for (int i = 0; i < VShare<D>::kWords; ++i) {
                    uint32_t r[4];
                    packed_octet(vs.w[i], vs.s[i >> 2], vs.z[i >> 2], r);
                    tc::st_shared_v4(vdst + s * L::KV_TILE + i * 16 * 128, r[0], r[1], r[2], r[3]);
                }
                // widened codes are visible to the tensor core before the warp arrives
                tc::fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
                    tc::mbar_arrive(&bars->k_full[s]);
                    tc::mbar_arrive(&bars->v_full[s]);
                }
                bool ok = true;
                if (t == 0 && records < n_hist) {
                    // the stage of a record that every producer warp has read by now, or soon
                    ok = tc::mbar_wait(&bars->r_empty[rs], (j / kRecStages) & 1, abort, a.status);
                    if (ok) fetch();
                }
                if (!__all_sync(0xffffffffu, ok)) break;
            } else {
                seg_tile(smem + L::K + s * L::KV_TILE, &tm_ks, j, &bars->k_full[s]);
                seg_tile(smem + L::V + s * L::KV_TILE, &tm_vs, j, &bars->v_full[s]);
            }
            issued = j + 1;
        }
    } else {
        // -------------------------------------------------------------- softmax / epilogue
        const int h = (warp - kSoftmax0) >> 2;  // M half
        const int quad = warp & 3;               // TMEM lane quadrant this warp may access
        const int r = quad * 32 + lane;          // row within the half = TMEM lane
        const int hh = 2 * h + (r >> 6);         // head within the group
        const int i = r & 63;                    // query row within the block
        const uint32_t lane_addr = (uint32_t)(quad * 32) << 16;
        const uint32_t o_addr = tmem + lane_addr + 128 * h;
        float m_run = -INFINITY, l_run = 0.f;
        bool ok = true;
        for (int j = 0; j < n_tiles; ++j) {
            const int bb = j & 1;
            // tcgen05.ld/st below are warp-collective: keep every decision warp-uniform
            if (!__all_sync(0xffffffffu, tc::mbar_wait(&bars->s_full[h][bb], (j >> 1) & 1, abort, a.status))) {
                ok = false;
                break;
            }
            tc::fence_after_sync();
            uint32_t sr[64];
            {
                uint32_t (&lo)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sr[0]);
                uint32_t (&hi)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sr[32]);
                const uint32_t s_addr = tmem + lane_addr + 256 + 128 * h + 64 * bb;
                tc::tmem_ld32(s_addr, lo);
                tc::tmem_ld32(s_addr + 32, hi);
                tc::tmem_wait_ld();
            }
            float x[64];
            const bool diag = (j == n_tiles - 1);  // the local tile of this block (warp-uniform)
#pragma unroll
            for (int c = 0; c < 64; ++c) x[c] = __uint_as_float(sr[c]);
            if (diag) {
#pragma unroll
                for (int c = 0; c < 64; ++c)
                    if (c > i) x[c] = -INFINITY;
            }
            // row max of the raw scores (the scale is positive), 4 chains of three-way maxima
            float mpart[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                mpart[c] = x[c];
#pragma unroll
                for (int e = c + 4; e < TILE; e += 8)
                    mpart[c] = e + 4 < TILE ? fmaxf(fmaxf(mpart[c], x[e]), x[e + 4]) : fmaxf(mpart[c], x[e]);
            }
            const float mx = fmaxf(fmaxf(mpart[0], mpart[1]), fmaxf(mpart[2], mpart[3])) * a.scale_log2;
            // Lazy rescaling: the reference max only moves when the row max grows by
            // more than kRescaleLog2, so P stays <= 2^kRescaleLog2 and O is rescaled
            // in TMEM only on those (rare) tiles.
            const bool grow = mx > m_run + kRescaleLog2;
            const float m_use = grow ? mx : m_run;
            const float alpha = grow ? tc::ex2(m_run - m_use) : 1.f;
            // a row with no unmasked key yet keeps m = -inf; its p must come out 0, not NaN
            const float m_sub = m_use == -INFINITY ? 0.f : m_use;
            // p = 2^(s * log2(e)/sqrt(D) - m), two elements per FMA and sum instruction
            float sp[4][2];
#pragma unroll
            for (int c = 0; c < TILE; c += 2) {
                fma2(x[c], x[c + 1], a.scale_log2, -m_sub);
                x[c] = tc::ex2(x[c]);
                x[c + 1] = tc::ex2(x[c + 1]);
                float (&q)[2] = sp[(c >> 1) & 3];
                if (c < 8) {
                    q[0] = x[c];
                    q[1] = x[c + 1];
                } else {
                    add2(q[0], q[1], x[c], x[c + 1]);
                }
            }
            const float sum = ((sp[0][0] + sp[1][0]) + (sp[2][0] + sp[3][0])) +
                              ((sp[0][1] + sp[1][1]) + (sp[2][1] + sp[3][1]));
            l_run = l_run * alpha + sum;
            const int pb = j & 1;
            // a rescale needs O complete up to tile j-1 (PV(j-1) done) before PV(j) adds to it;
            // rows that keep their reference max have alpha == 1, an exact no-op
            if (j >= 1 && __any_sync(0xffffffffu, grow)) {
                if (!__all_sync(0xffffffffu, tc::mbar_wait(&bars->o_done[h][pb ^ 1], ((j - 1) >> 1) & 1, abort,
                                                            a.status))) {
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t o[32];
                    tc::tmem_ld32(o_addr + c0, o);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
                    tc::tmem_st32(o_addr + c0, o);
                }
                tc::tmem_wait_st();
            }
            m_run = m_use;
            // P as bf16 pairs over the first 32 columns of this tile's S buffer (already
            // read into registers); PV reads it from there as its A operand, and bf16 products
            // take no wider one: outputs are 2.3e-3 in norm off those of 64 bits, 1.7e-3 with P
            // in fp32 (their own rounding).  The row sum is of the unrounded P.
            {
                uint32_t pk[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) pk[c] = tc::pack_bf16(x[2 * c], x[2 * c + 1]);
                tc::tmem_st32(tmem + lane_addr + 256 + 128 * h + 64 * pb, pk);
                tc::tmem_wait_st();
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars->p_full[h][pb]);
            if (NH == 2 && warp == kSoftmax0 && lane == 0) *reinterpret_cast<volatile int *>(&bars->sm0_tiles) = j + 1;
        }
        if (ok && __all_sync(0xffffffffu, tc::mbar_wait(&bars->o_done[h][(n_tiles - 1) & 1],
                                                        ((n_tiles - 1) >> 1) & 1, abort, a.status))) {
            tc::fence_after_sync();
            depend_next();
            const bool write = hh < a.hc;  // rows 64..127 repeat the head when HC = 1
            const long long row = ((long long)(b * a.n_q_heads + h0 + (write ? hh : 0))) * a.seg_len + m * TILE + i;
            const float inv_l = 1.f / l_run;
            // the rows go out through this half's Q tile, which its last product has read: a
            // thread's 16-byte pieces in the swizzled layout, then two TMA stores per warp of
            // 32 rows (76.0 -> 74.5 us on the 16K segment against stores from the registers)
            uint8_t *stage = smem + L::Q + h * L::Q_HALF;
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
                uint32_t o[32];
                tc::tmem_ld32(o_addr + c0, o);
                tc::tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 32; c += 8) {
                    uint32_t v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[e] = tc::pack_bf16(__uint_as_float(o[c + 2 * e]) * inv_l,
                                             __uint_as_float(o[c + 2 * e + 1]) * inv_l);
                    const uint32_t row = tc::smem_u32(stage) + (c0 >> 6) * (128 * 128) + r * 128;
                    const int piece = (c0 & 63) / 8 + c / 8;
                    tc::st_shared_v4(row + ((piece ^ (r & 7)) << 4), v[0], v[1], v[2], v[3]);
                }
            }
            tc::fence_proxy_async();
            __syncwarp();
            if (write && lane == 0) {
                const int orow = (b * a.n_q_heads + h0 + hh) * a.seg_len + m * TILE + (i & 32);
                for (int c = 0; c < D / 64; ++c)
                    tma_store_2d(&tm_o, stage + c * (128 * 128) + quad * (32 * 128), 64 * c, orow);
                bulk_commit();
                bulk_wait_all();
            }
            __syncwarp();
            if (write) a.lse[row] = (m_run + __log2f(l_run)) * 0.69314718055994530942f;
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (*abort) {
        // a wait gave up: let the copies and UMMAs still in flight finish before
        // shared memory and TMEM are released
        int never = 0;
        if (warp == kProd0 && lane == 0) {
            // stages whose segment tiles this thread sent for last; their barriers complete
            // once the other producer warps have arrived too, which an aborting one may not
            // have: the wait is bounded
            for (int j = issued - NSTAGE < n_hist ? n_hist : issued - NSTAGE; j < issued; ++j) {
                tc::mbar_wait(&bars->k_full[j % NSTAGE], (j / NSTAGE) & 1, &never, a.status, 1ll << 28);
                tc::mbar_wait(&bars->v_full[j % NSTAGE], (j / NSTAGE) & 1, &never, a.status, 1ll << 28);
            }
            for (int j = records < kRecStages ? 0 : records - kRecStages; j < records; ++j)
                tc::mbar_wait(&bars->r_full[j % kRecStages], (j / kRecStages) & 1, &never, a.status, 1ll << 28);
            tc::mbar_wait(&bars->q_full, 0, &never, a.status, 1ll << 28);
        }
        if (warp < kIssueWarps && (warp >> 1) < NH) {
            // the lane that issued this warp's MMAs commits and waits for them
            if (tc::elect_one()) {
                tc::mma_commit(&bars->drain[warp]);
                tc::mbar_wait(&bars->drain[warp], 0, &never, a.status, 1ll << 28);
            }
        }
        __syncwarp();
        tc::fence_after_sync();
        __syncthreads();
    }
    if (warp == 0) {
        __syncwarp();
        tc::tmem_dealloc<512>(tmem);
    }
}

template <int D, int NH>
hga_status_t launch_nh(const hga_params_t &p, const void *q, const uint8_t *hist, int cap, const void *ks,
                       const void *vs, const int32_t *idx, void *out, float *lse, unsigned *status,
                       cudaStream_t stream) {
    CUtensorMap mq, mks, mvs, mo;
    const long long n_bg = (long long)p.batch * p.n_kv_heads;
    const unsigned long long seg_rows = (unsigned long long)((n_bg - 1) * p.seg_head_stride + p.seg_len);
    const unsigned long long q_rows = (unsigned long long)p.batch * p.n_q_heads * p.seg_len;
    if (!tma_rows_map(&mq, q, q_rows, 64, D) || !tma_rows_map(&mo, out, q_rows, 32, D) ||
        !tma_rows_map(&mks, ks, seg_rows, 64, D) || !tma_rows_map(&mvs, vs, seg_rows, 64, D)) {
        record_error("hga_attn_fwd_packed: TMA tensor map encoding failed");
        return HGA_ERR_UNSUPPORTED;
    }
    const int nqb = p.seg_len / p.q_block;
    const int G = p.n_q_heads / p.n_kv_heads;
    FwdPackedArgs a;
    a.hc = NH == 2 ? 4 : (G % 2 == 0 ? 2 : 1);
    a.n_sub = G / a.hc;
    a.batch = p.batch;
    a.n_q_heads = p.n_q_heads;
    a.n_kv_heads = p.n_kv_heads;
    a.seg_len = p.seg_len;
    a.topk = p.topk;
    a.n_hist_chunks = p.n_hist_chunks;
    a.seg_stride = p.seg_head_stride;
    a.cap = cap;
    a.qb0 = p.qblock_end > 0 ? p.qblock_begin : 0;
    a.n_blocks = (p.qblock_end > 0 ? p.qblock_end : nqb) - a.qb0;
    a.hist = hist;
    a.idx = idx;
    a.lse = lse;
    a.status = status;
    a.scale_log2 = (float)(1.4426950408889634 / __builtin_sqrt((double)D));
    auto kern = attn_fwd_packed_kernel<D, NH>;
    cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void *>(kern), (int)Smem<D, NH>::ALLOC);
    if (e != cudaSuccess) return record_cuda(e);
    const unsigned grid = (unsigned)(a.n_blocks * n_bg * a.n_sub);
    // An SM runs one CTA at a time, and grid % SMs of the SMs get one more than the others.
    // Longest first alone, those end with a whole short block that nothing else runs beside;
    // from two CTAs an SM on they take it at the start instead.  us without / with, top-16 of 224
    // chunks: 320 CTAs 109.7 / 96.5, 384 131.6 / 124.0, 448 171.6 / 154.6, 512 202.7 / 186.7, 640
    // 294.5 / 291.7; top-4 of 64, 384 CTAs 68.9 / 65.0; the last 128K segment (512) 265 / 254.  Below
    // it gains nothing: 160 CTAs 48.6 / 48.4, 224 66.2 / 66.6, 256 74.5 / 76.
    const unsigned sms = (unsigned)sm_count();
    a.n_first = grid >= 2 * sms ? (int)(grid % sms) : 0;
    return record_cuda(launch_dependent(kern, grid, 32 * (kIssueWarps + 4 * NH + kProdWarps), Smem<D, NH>::ALLOC, 1,
                                        stream, mq, mks, mvs, mo, a));
}

}  // namespace

bool attn_fwd_packed_shape(const hga_params_t &p) {
    return p.dtype == HGA_BF16 && (p.head_dim == 64 || p.head_dim == 128) && p.chunk == 64 && p.q_block == 64;
}

bool attn_fwd_packed_supported(const hga_params_t &p) {
    if (!attn_fwd_packed_shape(p)) return false;
    // TMA row coordinates are 32-bit (queries and segment; the history is not read by TMA)
    if ((long long)p.batch * p.n_kv_heads * p.seg_head_stride >= (1ll << 31) ||
        (long long)p.batch * p.n_q_heads * p.seg_len >= (1ll << 31))
        return false;
    return tma_encoder_available();
}

hga_status_t launch_attn_fwd_packed(const hga_params_t &p, const void *q, const uint8_t *hist, int cap,
                                    const void *ks, const void *vs, const int32_t *idx, void *out, float *lse,
                                    unsigned *status, cudaStream_t stream) {
    const bool two = p.n_q_heads / p.n_kv_heads % 4 == 0;  // halves of two heads
    auto f = p.head_dim == 128 ? (two ? launch_nh<128, 2> : launch_nh<128, 1>)
                               : (two ? launch_nh<64, 2> : launch_nh<64, 1>);
    return f(p, q, hist, cap, ks, vs, idx, out, lse, status, stream);
}

}  // namespace hga
