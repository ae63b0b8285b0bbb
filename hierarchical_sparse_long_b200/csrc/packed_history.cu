// Packing closed chunks into 4-bit records at detach time, and reading them back.
//
// "Long-Context Fine-Tuning with Limited VRAM", technical summary section 2.2:
// detached history is read, never differentiated, and its memory grows with the
// context; a 4-bit record (packed.cuh) is 72 D bytes against 256 D in bf16.
//
// Grid of a group with extremes mn, mx (K: a channel's 64 tokens, V: 64 channels of a
// token), c nearest to the value, ties to even:
//   s = bf16(fl(fl(mx - mn) / 15)), 0 below 2^-100
//   z = bf16(fl(mn - 16 s)),   c = clamp(rne((x - z) / s) - 16, 0, 15), 0 where s = 0
// s and z are rounded first and the codes chosen for the rounded grid, so their
// rounding moves the grid and not the choice.  s = z = NaN when the group's sum is not
// finite (a NaN or an infinity in it) or s or z is not: its values read as NaN.
//
// pack is bound by HBM: K and V are read once (the summaries come from the same read),
// and 0.28 of their bytes written.  One 256-thread CTA takes a chunk, all 32 KiB of its
// loads in flight; K's extremes and sums cross threads through shared memory, V's stay
// in the lanes of a row, and V's codes are turned there from token to channel order.
#include <cfloat>

#include "packed.cuh"

namespace hga {

namespace {

constexpr int kChunk = 64;
constexpr int kThreads = 256;

struct Grid {
    float s, z;
};

__device__ __forceinline__ float bf16_round(float x) { return __bfloat162float(__float2bfloat16_rn(x)); }

__device__ __forceinline__ Grid make_grid(float mn, float mx, float sum) {
    Grid g;
    g.s = bf16_round(__fdiv_rn(mx - mn, 15.f));
    if (g.s < 0x1p-100f) g.s = 0.f;
    g.z = bf16_round(fmaf(-16.f, g.s, mn));
    // fabsf(NaN) <= FLT_MAX is false
    if (!(fabsf(sum) <= FLT_MAX) || !(fabsf(g.s) <= FLT_MAX) || !(fabsf(g.z) <= FLT_MAX))
        g.s = g.z = __int_as_float(0x7FC00000);
    return g;
}

// The code of x on grid g; inv = 1 / s.  t * inv is within 2^-22 of the quotient
// relatively (below 2^-17 in all), so unless it lies that close to a border its
// nearest integer is the quotient's; those that do are decided in 64 bits.
__device__ __forceinline__ uint32_t code_of(float x, const Grid &g, float inv) {
    const float q = (x - g.z) * inv;
    float k = rintf(q);
    if (fabsf(fabsf(q - k) - 0.5f) < 0x1p-15f) k = (float)rint(((double)x - (double)g.z) / (double)g.s);
    // a NaN grid compares false both ways and becomes code 0
    return k > 16.f ? (uint32_t)(fminf(k, 31.f) - 16.f) : 0u;
}

__device__ __forceinline__ float grid_inv(const Grid &g) { return g.s > 0.f ? 1.f / g.s : 0.f; }

__device__ __forceinline__ uint16_t bf16_bits(float x) {
    const __nv_bfloat16 b = __float2bfloat16_rn(x);
    return *reinterpret_cast<const uint16_t *>(&b);
}

// Thread (col, slot) owns VEC channels of the rows slot, slot + NSLOT, ...: the split of
// summaries_kernel, whose sums are repeated here in the same order bit for bit.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) pack_kernel(const T *__restrict__ k, const T *__restrict__ v,
                                                        long long head_stride, int n_chunks, int first_chunk,
                                                        uint8_t *__restrict__ hist, long long cap,
                                                        float *__restrict__ summ, long long summ_cap) {
    using P = Packed<D>;
    constexpr int VEC = Vec16<T>::N;
    constexpr int LPR = D / VEC;
    constexpr int NSLOT = kThreads / LPR;
    constexpr int ROWS = kChunk / NSLOT;
    constexpr int CS = D + 4;  // row stride of the staged V codes, bytes
    __shared__ float part[3][NSLOT][D + 1];
    __shared__ Grid kgrid[D];
    __shared__ __align__(16) uint8_t vcodes[kChunk * CS];
    const int tid = threadIdx.x;
    const long long slice = blockIdx.x / n_chunks;
    const int j = (int)(blockIdx.x % n_chunks);
    const int lane_col = tid % LPR, slot = tid / LPR;
    const int col = lane_col * VEC;
    const long long row0 = slice * head_stride + (long long)j * kChunk;
    uint8_t *rec = hist + (slice * cap + first_chunk + j) * P::kRecord;

    float x[ROWS][VEC], y[ROWS][VEC];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) Vec16<T>::load(k + (row0 + slot + r * NSLOT) * D + col, x[r]);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) Vec16<T>::load(v + (row0 + slot + r * NSLOT) * D + col, y[r]);

    // K: extremes and sum of every channel
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        float sum = 0.f, mn = x[0][e], mx = x[0][e];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            sum += x[r][e];
            mn = fminf(mn, x[r][e]);
            mx = fmaxf(mx, x[r][e]);
        }
        part[0][slot][col + e] = sum;
        part[1][slot][col + e] = mn;
        part[2][slot][col + e] = mx;
    }
    __syncthreads();
    if (tid < D) {
        float sum = 0.f, mn = part[1][0][tid], mx = part[2][0][tid];
#pragma unroll
        for (int s = 0; s < NSLOT; ++s) {
            sum += part[0][s][tid];
            mn = fminf(mn, part[1][s][tid]);
            mx = fmaxf(mx, part[2][s][tid]);
        }
        const Grid g = make_grid(mn, mx, sum);
        kgrid[tid] = g;
        uint16_t *gs = reinterpret_cast<uint16_t *>(rec + P::kGridOff);
        gs[tid] = bf16_bits(g.s);
        gs[D + tid] = bf16_bits(g.z);
        if (summ) summ[(slice * summ_cap + first_chunk + j) * D + tid] = sum / (float)kChunk;
    }

    // V: the grid of every token and 64 channels, from the lanes that hold them
    constexpr int GL = 64 / VEC;  // lanes per group
    uint16_t *vs = reinterpret_cast<uint16_t *>(rec + P::kPart + P::kGridOff);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        float sum = 0.f, mn = y[r][0], mx = y[r][0];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            sum += y[r][e];
            mn = fminf(mn, y[r][e]);
            mx = fmaxf(mx, y[r][e]);
        }
#pragma unroll
        for (int o = GL / 2; o; o >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        }
        const Grid g = make_grid(mn, mx, sum);
        const float inv = grid_inv(g);
        const int row = slot + r * NSLOT;
        if (lane_col % GL == 0) {
            vs[(col / 64) * kChunk + row] = bf16_bits(g.s);
            vs[D + (col / 64) * kChunk + row] = bf16_bits(g.z);
        }
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
            uint32_t w = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) w |= code_of(y[r][e + i], g, inv) << (8 * i);
            *reinterpret_cast<uint32_t *>(vcodes + row * CS + col + e) = w;
        }
    }
    __syncthreads();

    // K codes: a word holds the channels of one thread (bf16) or of a lane pair (fp32)
    uint32_t kw[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) kw[r] = 0;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const Grid g = kgrid[col + e];
        const float inv = grid_inv(g);
        const int el = (col + e) & 7;
        const int sh = 4 * (el >> 1) + 16 * (el & 1);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) kw[r] |= code_of(x[r][e], g, inv) << sh;
    }
    uint32_t *kcodes = reinterpret_cast<uint32_t *>(rec);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        if (VEC == 4) kw[r] |= __shfl_xor_sync(0xffffffffu, kw[r], 1);
        if (VEC == 8 || (lane_col & 1) == 0) kcodes[(slot + r * NSLOT) * (D / 8) + col / 8] = kw[r];
    }

    // V codes: four channels x eight tokens per step, turned in registers
    uint32_t *vw = reinterpret_cast<uint32_t *>(rec + P::kPart);
    for (int i = tid; i < 2 * D; i += kThreads) {
        const int w = i % 8, c4 = i / 8;
        uint32_t t[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) t[u] = *reinterpret_cast<const uint32_t *>(vcodes + (8 * w + u) * CS + 4 * c4);
        // bytes of a word: tokens 0 2 | 4 6 | 1 3 | 5 7, for each of the four channels
        const uint32_t b0 = t[0] | t[2] << 4, b1 = t[4] | t[6] << 4, b2 = t[1] | t[3] << 4, b3 = t[5] | t[7] << 4;
        const uint32_t lo01 = __byte_perm(b0, b1, 0x5140), hi01 = __byte_perm(b0, b1, 0x7362);
        const uint32_t lo23 = __byte_perm(b2, b3, 0x5140), hi23 = __byte_perm(b2, b3, 0x7362);
        vw[(4 * c4 + 0) * 8 + w] = __byte_perm(lo01, lo23, 0x5410);
        vw[(4 * c4 + 1) * 8 + w] = __byte_perm(lo01, lo23, 0x7632);
        vw[(4 * c4 + 2) * 8 + w] = __byte_perm(hi01, hi23, 0x5410);
        vw[(4 * c4 + 3) * 8 + w] = __byte_perm(hi01, hi23, 0x7632);
    }
}

__device__ __forceinline__ void store8(__nv_bfloat16 *p, const uint32_t (&r)[4]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(r[0], r[1], r[2], r[3]);
}
__device__ __forceinline__ void store8(float *p, const uint32_t (&r)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
        *reinterpret_cast<float4 *>(p + 4 * i) =
            make_float4(__uint_as_float(r[2 * i] << 16), __uint_as_float(r[2 * i] & 0xFFFF0000u),
                        __uint_as_float(r[2 * i + 1] << 16), __uint_as_float(r[2 * i + 1] & 0xFFFF0000u));
}

__device__ __forceinline__ void load4(const void *p, uint32_t (&r)[4]) {
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    r[0] = v.x;
    r[1] = v.y;
    r[2] = v.z;
    r[3] = v.w;
}

// One CTA per record, bound by the bytes it writes.  K words are 8 channels of a token,
// one 16-byte store (bf16) each; a V thread turns 8 channels x 8 tokens in registers.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) unpack_kernel(const uint8_t *__restrict__ hist, long long cap,
                                                          int first_chunk, int n_chunks, T *__restrict__ k,
                                                          T *__restrict__ v, long long head_stride) {
    using P = Packed<D>;
    constexpr int OPR = D / 8;
    const int tid = threadIdx.x;
    const long long slice = blockIdx.x / n_chunks;
    const int j = (int)(blockIdx.x % n_chunks);
    const uint8_t *rec = hist + (slice * cap + first_chunk + j) * P::kRecord;
    const long long row0 = slice * head_stride + (long long)j * kChunk;
    if (tid < kThreads / 2) {
        const int o = tid % OPR;
        uint32_t s[4], z[4], r[4];
        load4(rec + P::kGridOff + 16 * o, s);
        load4(rec + P::kGridOff + P::kGridHalf + 16 * o, z);
#pragma unroll
        for (int u = 0; u < kChunk * OPR / (kThreads / 2); ++u) {
            const int row = tid / OPR + u * (kThreads / 2 / OPR);
            packed_octet(reinterpret_cast<const uint32_t *>(rec)[row * OPR + o], s, z, r);
            store8(k + (row0 + row) * D + 8 * o, r);
        }
    } else {
        const uint8_t *vr = rec + P::kPart;
        for (int i = tid - kThreads / 2; i < D; i += kThreads / 2) {  // OPR octets of channels x 8 of tokens
            const int o = i % OPR, w = i / OPR;
            const uint8_t *grid = vr + P::kGridOff + (o / 8) * 2 * kChunk + 16 * w;
            uint32_t s[4], z[4], r[8][4];
            load4(grid, s);
            load4(grid + P::kGridHalf, z);
#pragma unroll
            for (int c = 0; c < 8; ++c)
                packed_octet(reinterpret_cast<const uint32_t *>(vr)[(8 * o + c) * 8 + w], s, z, r[c]);
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                uint32_t out[4];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    out[c] = __byte_perm(r[2 * c][t / 2], r[2 * c + 1][t / 2], (t & 1) ? 0x7632 : 0x5410);
                store8(v + (row0 + 8 * w + t) * D + 8 * o, out);
            }
        }
    }
}

template <typename T, int D>
hga_status_t pack_t(const void *k, const void *v, long long head_stride, long long slices, int first_chunk,
                    int n_chunks, uint8_t *hist, int cap, float *summ, int summ_cap, cudaStream_t stream) {
    pack_kernel<T, D><<<(unsigned)(slices * n_chunks), kThreads, 0, stream>>>(
        static_cast<const T *>(k), static_cast<const T *>(v), head_stride, n_chunks, first_chunk, hist, cap, summ,
        summ_cap);
    return record_cuda(cudaGetLastError());
}

template <typename T, int D>
hga_status_t unpack_t(const uint8_t *hist, int cap, long long slices, int first_chunk, int n_chunks, void *k, void *v,
                      long long head_stride, cudaStream_t stream) {
    unpack_kernel<T, D><<<(unsigned)(slices * n_chunks), kThreads, 0, stream>>>(
        hist, cap, first_chunk, n_chunks, static_cast<T *>(k), static_cast<T *>(v), head_stride);
    return record_cuda(cudaGetLastError());
}

}  // namespace

hga_status_t launch_pack_history(const void *k, const void *v, long long head_stride, long long slices, int head_dim,
                                 int first_chunk, int n_chunks, hga_dtype_t dtype, uint8_t *hist, int cap, float *summ,
                                 int summ_cap, cudaStream_t stream) {
    auto f = dtype == HGA_BF16 ? (head_dim == 128 ? pack_t<__nv_bfloat16, 128> : pack_t<__nv_bfloat16, 64>)
                               : (head_dim == 128 ? pack_t<float, 128> : pack_t<float, 64>);
    return f(k, v, head_stride, slices, first_chunk, n_chunks, hist, cap, summ, summ_cap, stream);
}

hga_status_t launch_unpack_history(const uint8_t *hist, int cap, long long slices, int head_dim, int first_chunk,
                                   int n_chunks, hga_dtype_t dtype, void *k, void *v, long long head_stride,
                                   cudaStream_t stream) {
    auto f = dtype == HGA_BF16 ? (head_dim == 128 ? unpack_t<__nv_bfloat16, 128> : unpack_t<__nv_bfloat16, 64>)
                               : (head_dim == 128 ? unpack_t<float, 128> : unpack_t<float, 64>);
    return f(hist, cap, slices, first_chunk, n_chunks, k, v, head_stride, stream);
}

}  // namespace hga
