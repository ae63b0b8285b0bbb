// From a layer's projections to the attention's inputs, and back.
//
// "Long-Context Fine-Tuning with Limited VRAM", technical summary section 2.1,
// takes queries, keys and values per head and position as given; this file is
// the step that gives them: per-head RMS norm of q and k, the position
// rotation, and the turn from token-major projection rows to the head-major
// tensors that every attention call reads.
//
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r w
//   y_i       = n_i c_i - n_{i+R/2} s_i        i < R/2, (c, s) of the token's
//   y_{i+R/2} = n_{i+R/2} c_i + n_i s_i        position; dims >= R: y = n
// and with dn the transposed rotation of dy, xh = x r, g = dn w:
//   dx = r (g - xh mean(g xh)),   dw = sum over rows of dn xh.
//
// Both directions are bound by HBM: each row is read and written once, a
// token's cos / sin row is read by the CTAs of its heads (L2 after the first).
// A row of D elements belongs to D / (2 VEC) lanes of 16-byte vectors, each
// lane holding a rotation pair of vectors (i, i + R/2) -- or two unrotated
// ones past R -- so the rotation stays inside a thread and only the mean
// crosses lanes.  A CTA takes a few heads (gridDim.y) of a run of tokens: its
// reads are whole 128-byte lines of token rows, its writes consecutive rows of
// a head.
#include "common.cuh"

namespace hga {

namespace {

constexpr int kThreads = 128;
constexpr int kHeads = 4;  // heads per thread of a long call

struct NormRopeArgs {
    const void *x[3];  // q, k, v projections
    const void *w[2];
    const float *table;
    const int32_t *positions;
    void *y[3];
    const float *dy[3];
    void *dx[3];
    float *partial;  // [gridDim.y of q and k][gridDim.x][D]
    float *dw[2];
    unsigned *status;
    long long x_stride[3];  // elements between tokens
    long long pos0, n_pos, kv_stride;
    int batch, seq_len, heads[2], rot;  // heads: q, kv
    int groups[2];                      // head groups of q, of k (= of v)
    float eps;
};

template <typename T> __device__ __forceinline__ void store_vec(T *p, const float *v);
template <> __device__ __forceinline__ void store_vec<float>(float *p, const float *v) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
template <> __device__ __forceinline__ void store_vec<__nv_bfloat16>(__nv_bfloat16 *p, const float *v) {
    uint4 u;
    uint32_t *w = &u.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    *reinterpret_cast<uint4 *>(p) = u;
}
template <int N> __device__ __forceinline__ void load_f32(const float *p, float *v) {
#pragma unroll
    for (int i = 0; i < N; i += 4) Vec16<float>::load(p + i, v + i);
}

// Sum over the L lanes of a row.
template <int L> __device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = L / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Where a CTA's heads lie: kind 0 q, 1 k, 2 v, and its first head.
__device__ __forceinline__ int cta_kind(const NormRopeArgs &a, int heads_per, int &h0) {
    int gy = (int)blockIdx.y, kind = 0;
    if (gy >= a.groups[0]) {
        gy -= a.groups[0];
        kind = 1;
        if (gy >= a.groups[1]) {
            gy -= a.groups[1];
            kind = 2;
        }
    }
    h0 = gy * heads_per;
    return kind;
}

// Position of token t (b * S + i), or -1 for a padding row (and, flagged, for a
// position that the table does not hold).
__device__ __forceinline__ long long token_pos(const NormRopeArgs &a, long long t) {
    if (!a.positions) return a.pos0 + t % a.seq_len;
    const int p = a.positions[t];
    if (p >= 0 && (a.rot == 0 || p < a.n_pos)) return p;
    if (p != -1) atomicOr(a.status, kDevBadIndex);
    return -1;
}

// The two vectors of a row that lane l holds, and cos / sin of their pairs.
template <int VEC> __device__ __forceinline__ bool lane_vectors(const NormRopeArgs &a, int l, int &e0, int &e1) {
    const int half = a.rot / (2 * VEC);
    const bool rotated = l < half;
    e0 = rotated ? l * VEC : a.rot + (l - half) * 2 * VEC;
    e1 = rotated ? e0 + a.rot / 2 : e0 + VEC;
    return rotated;
}

template <int VEC>
__device__ __forceinline__ void load_cs(const NormRopeArgs &a, long long pos, int e0, bool rotated, float *c,
                                        float *s) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        c[e] = 1.f;
        s[e] = 0.f;
    }
    if (rotated) {
        const float *row = a.table + pos * a.rot + e0;
        load_f32<VEC>(row, c);
        load_f32<VEC>(row + a.rot / 2, s);
    }
}

// HPT heads of one token per thread group.  Long calls take four, whose loads are in
// flight together and share the token's cos / sin and the weights; short ones take
// one, so that a single token's heads spread over more SMs.
template <typename T, int D, int HPT>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormRopeArgs a) {
    constexpr int VEC = Vec16<T>::N;
    constexpr int L = D / (2 * VEC);  // lanes per row
    int h0;
    const int kind = cta_kind(a, HPT, h0);
    const int n_heads = a.heads[kind > 0];
    const int l = threadIdx.x % L;
    const long long n_tok = (long long)a.batch * a.seq_len;
    const long long t = (long long)blockIdx.x * (kThreads / L) + threadIdx.x / L;
    const bool live = t < n_tok;
    const long long pos = live ? token_pos(a, t) : -1;
    int e0, e1;
    const bool rotated = lane_vectors<VEC>(a, l, e0, e1);

    float x[HPT][2][VEC];
    const T *src = static_cast<const T *>(a.x[kind]) + t * a.x_stride[kind];
#pragma unroll
    for (int h = 0; h < HPT; ++h)
        if (pos >= 0 && h0 + h < n_heads) {
            Vec16<T>::load(src + (h0 + h) * D + e0, x[h][0]);
            Vec16<T>::load(src + (h0 + h) * D + e1, x[h][1]);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[h][0][e] = x[h][1][e] = 0.f;
        }
    const long long b = t / a.seq_len, i = t % a.seq_len;
    const long long hs = kind == 0 ? a.seq_len : a.kv_stride;
    T *dst = static_cast<T *>(a.y[kind]);
    if (kind < 2) {
        float w[2][VEC], c[VEC], s[VEC];
        Vec16<T>::load(static_cast<const T *>(a.w[kind]) + e0, w[0]);
        Vec16<T>::load(static_cast<const T *>(a.w[kind]) + e1, w[1]);
        load_cs<VEC>(a, pos, e0, rotated && pos >= 0, c, s);
#pragma unroll
        for (int h = 0; h < HPT; ++h) {
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < VEC; ++e) sum = fmaf(x[h][0][e], x[h][0][e], fmaf(x[h][1][e], x[h][1][e], sum));
            const float r = rsqrtf(row_sum<L>(sum) * (1.f / D) + a.eps);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float n0 = x[h][0][e] * r * w[0][e], n1 = x[h][1][e] * r * w[1][e];
                x[h][0][e] = n0 * c[e] - n1 * s[e];
                x[h][1][e] = n1 * c[e] + n0 * s[e];
            }
        }
    }
    if (pos < 0) return;
#pragma unroll
    for (int h = 0; h < HPT; ++h)
        if (h0 + h < n_heads) {
            T *row = dst + ((b * n_heads + h0 + h) * hs + i) * D;
            store_vec<T>(row + e0, x[h][0]);
            store_vec<T>(row + e1, x[h][1]);
        }
}

// Gradients: dx of each row, and per CTA the sum over its rows of dn xh, which
// norm_rope_dw adds up in a fixed order (no atomics: the same inputs give the same bits).
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) norm_rope_bwd_kernel(const NormRopeArgs a) {
    constexpr int VEC = Vec16<T>::N;
    constexpr int L = D / (2 * VEC);
    constexpr int SLOTS = kThreads / L;  // tokens at once
    __shared__ float part[SLOTS][D + 4];
    int h0;
    const int kind = cta_kind(a, kHeads, h0);
    const int n_heads = a.heads[kind > 0];
    const int l = threadIdx.x % L, slot = threadIdx.x / L;
    const long long n_tok = (long long)a.batch * a.seq_len;
    int e0, e1;
    const bool rotated = lane_vectors<VEC>(a, l, e0, e1);
    float w[2][VEC], dw[2][VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[0][e] = dw[1][e] = 0.f;
    if (kind < 2) {
        Vec16<T>::load(static_cast<const T *>(a.w[kind]) + e0, w[0]);
        Vec16<T>::load(static_cast<const T *>(a.w[kind]) + e1, w[1]);
    }
    // every lane of a warp takes the same number of steps: the row sums are warp-wide
    for (long long t0 = (long long)blockIdx.x * SLOTS; t0 < n_tok; t0 += (long long)gridDim.x * SLOTS) {
        const long long t = t0 + slot;
        const bool live = t < n_tok;
        const long long pos = live ? token_pos(a, t) : -1;
        const long long b = t / a.seq_len, i = t % a.seq_len;
        const T *src = static_cast<const T *>(a.x[kind]) + t * a.x_stride[kind];
        T *dst = static_cast<T *>(a.dx[kind]) + t * a.x_stride[kind];
        float c[VEC], s[VEC];
        if (kind < 2) load_cs<VEC>(a, pos, e0, rotated && pos >= 0, c, s);
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
            const bool on = pos >= 0 && h0 + h < n_heads;
            float g[2][VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) g[0][e] = g[1][e] = 0.f;
            if (on) {
                const float *row = a.dy[kind] + ((b * n_heads + h0 + h) * (long long)a.seq_len + i) * D;
                load_f32<VEC>(row + e0, g[0]);
                load_f32<VEC>(row + e1, g[1]);
            }
            if (kind < 2) {
                float x[2][VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) x[0][e] = x[1][e] = 0.f;
                if (on) {
                    Vec16<T>::load(src + (h0 + h) * D + e0, x[0]);
                    Vec16<T>::load(src + (h0 + h) * D + e1, x[1]);
                }
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < VEC; ++e) sum = fmaf(x[0][e], x[0][e], fmaf(x[1][e], x[1][e], sum));
                const float r = rsqrtf(row_sum<L>(sum) * (1.f / D) + a.eps);
                float dot = 0.f;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float dn0 = g[0][e] * c[e] + g[1][e] * s[e];
                    const float dn1 = g[1][e] * c[e] - g[0][e] * s[e];
                    x[0][e] *= r;
                    x[1][e] *= r;
                    dw[0][e] = fmaf(dn0, x[0][e], dw[0][e]);
                    dw[1][e] = fmaf(dn1, x[1][e], dw[1][e]);
                    g[0][e] = dn0 * w[0][e];
                    g[1][e] = dn1 * w[1][e];
                    dot = fmaf(g[0][e], x[0][e], fmaf(g[1][e], x[1][e], dot));
                }
                dot = row_sum<L>(dot) * (1.f / D);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    g[0][e] = r * (g[0][e] - x[0][e] * dot);
                    g[1][e] = r * (g[1][e] - x[1][e] * dot);
                }
            }
            if (live && h0 + h < n_heads) {  // a padding row's gradient is zero
                store_vec<T>(dst + (h0 + h) * D + e0, g[0]);
                store_vec<T>(dst + (h0 + h) * D + e1, g[1]);
            }
        }
    }
    if (kind == 2) return;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        part[slot][e0 + e] = dw[0][e];
        part[slot][e1 + e] = dw[1][e];
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kThreads) {
        float sum = 0.f;
#pragma unroll
        for (int sl = 0; sl < SLOTS; ++sl) sum += part[sl][d];
        a.partial[((long long)blockIdx.y * gridDim.x + blockIdx.x) * D + d] = sum;
    }
}

// dw of q (blockIdx.y = 0) and k (1): the partials of its head groups, in order, in
// 64 bits.  A CTA takes 8 dims with 32 threads each (every 32nd partial, then a tree).
template <int D>
__global__ void __launch_bounds__(256) norm_rope_dw(const NormRopeArgs a, int grid_x) {
    __shared__ double part[32][8];
    const int kind = blockIdx.y, d = threadIdx.x % 8, slot = threadIdx.x / 8;
    const long long n = (long long)a.groups[kind] * grid_x;
    const float *p = a.partial + (kind ? (long long)a.groups[0] * grid_x * D : 0) + blockIdx.x * 8 + d;
    double sum = 0.0;
    for (long long i = slot; i < n; i += 32) sum += (double)p[i * D];
    part[slot][d] = sum;
    __syncthreads();
    if (slot == 0) {
        for (int i = 1; i < 32; ++i) sum += part[i][d];
        a.dw[kind][blockIdx.x * 8 + d] = (float)sum;
    }
}

// cos then sin of pos * theta^(-2 i / R): angles in 64 bits (a 32-bit angle of
// position 131,071 is off by up to 2^-8), rounded once.
__global__ void rope_table_kernel(double log_theta, int rot, long long n_pos, float *table) {
    const long long at = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const int half = rot / 2;
    if (at >= n_pos * half) return;
    const long long pos = at / half;
    const int i = (int)(at % half);
    double s, c;
    sincos((double)pos * exp(-log_theta * (2.0 * i / rot)), &s, &c);
    table[pos * rot + i] = (float)c;
    table[pos * rot + half + i] = (float)s;
}

NormRopeArgs make_args(const hga_proj_t &p, const void *q, const void *k, const void *v, const void *qw,
                       const void *kw, const float *table, long long n_pos, const int32_t *positions,
                       unsigned *status) {
    NormRopeArgs a = {};
    a.x[0] = q;
    a.x[1] = k;
    a.x[2] = v;
    a.w[0] = qw;
    a.w[1] = kw;
    a.table = table;
    a.positions = positions;
    a.status = status;
    a.x_stride[0] = p.q_token_stride;
    a.x_stride[1] = p.k_token_stride;
    a.x_stride[2] = p.v_token_stride;
    a.pos0 = p.first_pos;
    a.n_pos = n_pos;
    a.kv_stride = p.kv_head_stride;
    a.batch = p.batch;
    a.seq_len = p.seq_len;
    a.heads[0] = p.n_q_heads;
    a.heads[1] = p.n_kv_heads;
    a.rot = p.rotary_dim;
    a.eps = p.eps;
    return a;
}

void set_groups(NormRopeArgs &a, int heads_per) {
    for (int i = 0; i < 2; ++i) a.groups[i] = (a.heads[i] + heads_per - 1) / heads_per;
}

template <typename T, int D> hga_status_t launch_fwd(NormRopeArgs a, cudaStream_t stream) {
    constexpr int slots = kThreads / (D / (2 * Vec16<T>::N));
    const long long n_tok = (long long)a.batch * a.seq_len;
    const long long gx = (n_tok + slots - 1) / slots;
    set_groups(a, kHeads);
    if (gx * (a.groups[0] + 2 * a.groups[1]) >= 2 * sm_count()) {
        norm_rope_kernel<T, D, kHeads>
            <<<dim3((unsigned)gx, a.groups[0] + 2 * a.groups[1]), kThreads, 0, stream>>>(a);
    } else {
        set_groups(a, 1);
        norm_rope_kernel<T, D, 1><<<dim3((unsigned)gx, a.groups[0] + 2 * a.groups[1]), kThreads, 0, stream>>>(a);
    }
    return record_cuda(cudaGetLastError());
}

// CTAs along the tokens of the backward: four CTAs per SM over all head groups.
// A fixed number, so that the workspace size needs no device.
long long bwd_grid_x(const hga_proj_t &p) {
    const int lanes = p.head_dim / (p.dtype == HGA_FP32 ? 8 : 16);
    const int slots = kThreads / lanes;
    const long long steps = ((long long)p.batch * p.seq_len + slots - 1) / slots;
    const int groups = (p.n_q_heads + kHeads - 1) / kHeads + 2 * ((p.n_kv_heads + kHeads - 1) / kHeads);
    const long long want = (148 * 4 + groups - 1) / groups;
    return steps < want ? steps : want;
}

template <typename T, int D> hga_status_t launch_bwd(NormRopeArgs a, long long gx, cudaStream_t stream) {
    set_groups(a, kHeads);
    norm_rope_bwd_kernel<T, D><<<dim3((unsigned)gx, a.groups[0] + 2 * a.groups[1]), kThreads, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return record_cuda(e);
    norm_rope_dw<D><<<dim3(D / 8, 2), 256, 0, stream>>>(a, (int)gx);
    return record_cuda(cudaGetLastError());
}

}  // namespace

hga_status_t launch_rope_table(double theta, int rotary_dim, long long n_pos, float *table, cudaStream_t stream) {
    const long long n = n_pos * (rotary_dim / 2);
    rope_table_kernel<<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(log(theta), rotary_dim, n_pos, table);
    return record_cuda(cudaGetLastError());
}

hga_status_t launch_qk_norm_rope(const hga_proj_t &p, const void *q, const void *k, const void *v, const void *qw,
                                 const void *kw, const float *table, long long n_pos, const int32_t *positions,
                                 void *q_out, void *k_out, void *v_out, unsigned *status, cudaStream_t stream) {
    NormRopeArgs a = make_args(p, q, k, v, qw, kw, table, n_pos, positions, status);
    a.y[0] = q_out;
    a.y[1] = k_out;
    a.y[2] = v_out;
    if (p.dtype == HGA_BF16)
        return p.head_dim == 128 ? launch_fwd<__nv_bfloat16, 128>(a, stream) : launch_fwd<__nv_bfloat16, 64>(a, stream);
    return p.head_dim == 128 ? launch_fwd<float, 128>(a, stream) : launch_fwd<float, 64>(a, stream);
}

size_t qk_norm_rope_workspace_bytes(const hga_proj_t &p) {
    const size_t groups = (p.n_q_heads + kHeads - 1) / kHeads + (p.n_kv_heads + kHeads - 1) / kHeads;
    return groups * (size_t)bwd_grid_x(p) * p.head_dim * sizeof(float);
}

hga_status_t launch_qk_norm_rope_bwd(const hga_proj_t &p, const void *q, const void *k, const void *qw,
                                     const void *kw, const float *table, long long n_pos, const int32_t *positions,
                                     const float *dq, const float *dk, const float *dv, void *dq_in, void *dk_in,
                                     void *dv_in, float *dqw, float *dkw, float *ws, unsigned *status,
                                     cudaStream_t stream) {
    NormRopeArgs a = make_args(p, q, k, nullptr, qw, kw, table, n_pos, positions, status);
    a.dy[0] = dq;
    a.dy[1] = dk;
    a.dy[2] = dv;
    a.dx[0] = dq_in;
    a.dx[1] = dk_in;
    a.dx[2] = dv_in;
    a.partial = ws;
    a.dw[0] = dqw;
    a.dw[1] = dkw;
    const long long gx = bwd_grid_x(p);
    if (p.dtype == HGA_BF16)
        return p.head_dim == 128 ? launch_bwd<__nv_bfloat16, 128>(a, gx, stream)
                                 : launch_bwd<__nv_bfloat16, 64>(a, gx, stream);
    return p.head_dim == 128 ? launch_bwd<float, 128>(a, gx, stream) : launch_bwd<float, 64>(a, gx, stream);
}

}  // namespace hga
