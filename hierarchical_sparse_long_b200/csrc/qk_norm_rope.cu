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
// Both directions' floor is HBM: each row is read and written once, a token's cos / sin
// row is read by the CTAs of its heads (L2 after the first).  What they spend beyond it is
// latency (a row is loaded, reduced over its lanes and stored, with 20 resident warps an SM
// to overlap in the forward, 12 in the backward).  A row of D elements belongs to D / (2 VEC) lanes of 16-byte vectors, each
// lane holding a rotation pair of vectors (i, i + R/2) -- or two unrotated ones past R -- so
// the rotation stays inside a thread and only the mean crosses lanes.  A CTA takes a few
// heads (gridDim.y) of a run of tokens: its reads are whole 128-byte lines of token rows,
// its writes consecutive rows of a head.  2,048 tokens of 32 + 8 heads of 128 in bf16: forward
// 10.3 us (50 MB, 4.9 TB/s), backward 21.7 us (98 MB, 4.5 TB/s); with scalar arithmetic and
// loads behind the position's they took 16.6 and 33.1 us.
#include "common.cuh"
#include "dependent.cuh"

namespace hga {

namespace {

constexpr int kThreads = 128;
constexpr int kHeads = 4;  // heads per thread of a long call
constexpr int kBwdCtas = 3;  // CTAs per SM of the backward: 168 registers a thread

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

// A 16-byte vector as pairs of fp32, the operands of the two-element instructions.
template <typename T> struct Pairs {
    static constexpr int N = Vec16<T>::N / 2;
    float2 v[N];
    __device__ __forceinline__ static Pairs widen(const uint4 &u) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        Pairs p;
#pragma unroll
        for (int i = 0; i < N; ++i)
            p.v[i] = sizeof(T) == 2
                         ? make_float2(__uint_as_float(w[i % 4] << 16), __uint_as_float(w[i % 4] & 0xFFFF0000u))
                         : make_float2(__uint_as_float(w[2 * i % 4]), __uint_as_float(w[(2 * i + 1) % 4]));
        return p;
    }
    __device__ __forceinline__ static Pairs fill(float x) {
        Pairs p;
#pragma unroll
        for (int i = 0; i < N; ++i) p.v[i] = make_float2(x, x);
        return p;
    }
    __device__ __forceinline__ static Pairs load_f32(const float *src) {
        Pairs p;
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float4 f = *reinterpret_cast<const float4 *>(src + 2 * i);
            p.v[i] = make_float2(f.x, f.y);
            p.v[i + 1] = make_float2(f.z, f.w);
        }
        return p;
    }
    // rounded to T
    __device__ __forceinline__ void store(T *dst) const {
        uint4 u;
        uint32_t *w = &u.x;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (sizeof(T) == 2) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[i].x, v[i].y);
                w[i] = *reinterpret_cast<const uint32_t *>(&b);
            } else {
                w[2 * i] = __float_as_uint(v[i].x);
                w[2 * i + 1] = __float_as_uint(v[i].y);
            }
        }
        *reinterpret_cast<uint4 *>(dst) = u;
    }
};
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 minus(float2 x) { return make_float2(-x.x, -x.y); }

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

// cos and sin of a lane's pairs.
template <typename T> struct Turn {
    Pairs<T> c, s;
    __device__ __forceinline__ Turn(const NormRopeArgs &a, long long pos, int e0, bool rotated) {
        c = Pairs<T>::fill(1.f);
        s = Pairs<T>::fill(0.f);
        if (rotated) {
            const float *row = a.table + pos * a.rot + e0;
            c = Pairs<T>::load_f32(row);
            s = Pairs<T>::load_f32(row + a.rot / 2);
        }
    }
};

// 1 / sqrt(mean square + eps) of a row whose lane holds x0, x1.
template <typename T, int D> __device__ __forceinline__ float rms(const Pairs<T> &x0, const Pairs<T> &x1, float eps) {
    float2 sum = __fmul2_rn(x0.v[0], x0.v[0]);
#pragma unroll
    for (int i = 1; i < Pairs<T>::N; ++i) sum = __ffma2_rn(x0.v[i], x0.v[i], sum);
#pragma unroll
    for (int i = 0; i < Pairs<T>::N; ++i) sum = __ffma2_rn(x1.v[i], x1.v[i], sum);
    return rsqrtf(row_sum<D / (2 * Vec16<T>::N)>(sum.x + sum.y) * (1.f / D) + eps);
}

// HPT heads of one token per thread group.  Long calls take four, whose loads are in
// flight together and share the token's cos / sin and the weights; short ones take
// one, so that a single token's heads spread over more SMs.  The rows are asked for before
// the position is known (a padding row's are read and dropped): one latency less.  They are
// read once, as data to evict first, which leaves more of L2 to the outputs: 10.4 -> 10.3 us
// on the 2,048-token segment.
template <typename T, int D, int HPT>
__global__ void __launch_bounds__(kThreads, HPT == 1 ? 8 : 5) norm_rope_kernel(const NormRopeArgs a) {
    using Pr = Pairs<T>;
    constexpr int VEC = Vec16<T>::N;
    constexpr int L = D / (2 * VEC);  // lanes per row
    int h0;
    const int kind = cta_kind(a, HPT, h0);
    const int n_heads = a.heads[kind > 0];
    const int l = threadIdx.x % L;
    const long long n_tok = (long long)a.batch * a.seq_len;
    const long long t = (long long)blockIdx.x * (kThreads / L) + threadIdx.x / L;
    const bool live = t < n_tok;
    int e0, e1;
    const bool rotated = lane_vectors<VEC>(a, l, e0, e1);

    depend_wait();
    uint4 x[HPT][2];
    const T *src = static_cast<const T *>(a.x[kind]) + t * a.x_stride[kind] + h0 * D;
#pragma unroll
    for (int h = 0; h < HPT; ++h) {
        x[h][0] = x[h][1] = make_uint4(0u, 0u, 0u, 0u);
        if (live && h0 + h < n_heads) {
            x[h][0] = __ldcs(reinterpret_cast<const uint4 *>(src + h * D + e0));
            x[h][1] = __ldcs(reinterpret_cast<const uint4 *>(src + h * D + e1));
        }
    }
    const long long pos = live ? token_pos(a, t) : -1;
    const long long b = t / a.seq_len, i = t % a.seq_len;
    const long long hs = kind == 0 ? a.seq_len : a.kv_stride;
    T *dst = static_cast<T *>(a.y[kind]) + ((b * n_heads + h0) * hs + i) * D;
    if (kind == 2) {
        if (pos < 0) return;
#pragma unroll
        for (int h = 0; h < HPT; ++h)
            if (h0 + h < n_heads) {
                *reinterpret_cast<uint4 *>(dst + h * hs * D + e0) = x[h][0];
                *reinterpret_cast<uint4 *>(dst + h * hs * D + e1) = x[h][1];
            }
        return;
    }
    const T *wp = static_cast<const T *>(a.w[kind]);
    const Pr w0 = Pr::widen(*reinterpret_cast<const uint4 *>(wp + e0));
    const Pr w1 = Pr::widen(*reinterpret_cast<const uint4 *>(wp + e1));
    const Turn<T> turn(a, pos, e0, rotated && pos >= 0);
    depend_next();
#pragma unroll
    for (int h = 0; h < HPT; ++h) {
        Pr x0 = Pr::widen(x[h][0]), x1 = Pr::widen(x[h][1]);
        const float2 r = both(rms<T, D>(x0, x1, a.eps));
#pragma unroll
        for (int j = 0; j < Pr::N; ++j) {
            const float2 n0 = __fmul2_rn(__fmul2_rn(x0.v[j], r), w0.v[j]);
            const float2 n1 = __fmul2_rn(__fmul2_rn(x1.v[j], r), w1.v[j]);
            x0.v[j] = __ffma2_rn(n0, turn.c.v[j], minus(__fmul2_rn(n1, turn.s.v[j])));
            x1.v[j] = __ffma2_rn(n0, turn.s.v[j], __fmul2_rn(n1, turn.c.v[j]));
        }
        if (pos >= 0 && h0 + h < n_heads) {
            x0.store(dst + h * hs * D + e0);
            x1.store(dst + h * hs * D + e1);
        }
    }
}

// Gradients: dx of each row, and per CTA the sum over its rows of dn xh, which
// norm_rope_dw adds up in a fixed order (no atomics: the same inputs give the same bits).
// A thread's and a CTA's sums are 32 bits, the rest 64: the weights' gradients are off those of
// 64-bit sums by 1.2e-7 in norm for 2,048 tokens of 32 + 8 heads and by 3.4e-7 for 65,536 of
// 16 + 1 (rounding the result alone is 7e-8), and a thread has no registers for longer sums.
// Heads go in pairs, whose loads are in flight together; a head's are 96 bytes a lane.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, kBwdCtas) norm_rope_bwd_kernel(const NormRopeArgs a) {
    using Pr = Pairs<T>;
    constexpr int VEC = Vec16<T>::N;
    constexpr int L = D / (2 * VEC);
    constexpr int SLOTS = kThreads / L;  // tokens at once
    constexpr int HP = 2;
    __shared__ float part[SLOTS][D + 4];
    int h0;
    const int kind = cta_kind(a, kHeads, h0);
    const int n_heads = a.heads[kind > 0];
    const int l = threadIdx.x % L, slot = threadIdx.x / L;
    const long long n_tok = (long long)a.batch * a.seq_len;
    int e0, e1;
    const bool rotated = lane_vectors<VEC>(a, l, e0, e1);
    depend_wait();
    Pr dw0 = Pr::fill(0.f), dw1 = dw0;
    uint4 wr[2] = {};
    if (kind < 2) {
        wr[0] = *reinterpret_cast<const uint4 *>(static_cast<const T *>(a.w[kind]) + e0);
        wr[1] = *reinterpret_cast<const uint4 *>(static_cast<const T *>(a.w[kind]) + e1);
    }
    // every lane of a warp takes the same number of steps: the row sums are warp-wide
    for (long long t0 = (long long)blockIdx.x * SLOTS; t0 < n_tok; t0 += (long long)gridDim.x * SLOTS) {
        const long long t = t0 + slot;
        const bool live = t < n_tok;
        const long long b = t / a.seq_len, i = t % a.seq_len;
        const T *src = static_cast<const T *>(a.x[kind]) + t * a.x_stride[kind] + h0 * D;
        T *dst = static_cast<T *>(a.dx[kind]) + t * a.x_stride[kind] + h0 * D;
        const float *dy = a.dy[kind] + ((b * n_heads + h0) * (long long)a.seq_len + i) * D;
        const long long dy_head = (long long)a.seq_len * D;
        const long long pos = live ? token_pos(a, t) : -1;
        const Turn<T> turn(a, pos, e0, kind < 2 && rotated && pos >= 0);
#pragma unroll
        for (int hp = 0; hp < kHeads; hp += HP) {
            if (h0 + hp >= n_heads) break;
            Pr g0[HP], g1[HP];
            uint4 x[HP][2];
#pragma unroll
            for (int h = 0; h < HP; ++h) {
                g0[h] = g1[h] = Pr::fill(0.f);
                x[h][0] = x[h][1] = make_uint4(0u, 0u, 0u, 0u);
                if (pos >= 0 && h0 + hp + h < n_heads) {
                    g0[h] = Pr::load_f32(dy + (hp + h) * dy_head + e0);
                    g1[h] = Pr::load_f32(dy + (hp + h) * dy_head + e1);
                    if (kind < 2) {
                        x[h][0] = *reinterpret_cast<const uint4 *>(src + (hp + h) * D + e0);
                        x[h][1] = *reinterpret_cast<const uint4 *>(src + (hp + h) * D + e1);
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < HP; ++h) {
                if (kind < 2) {
                    Pr x0 = Pr::widen(x[h][0]), x1 = Pr::widen(x[h][1]);
                    const Pr w0 = Pr::widen(wr[0]), w1 = Pr::widen(wr[1]);
                    const float r = rms<T, D>(x0, x1, a.eps);
                    float2 dot2 = both(0.f);
#pragma unroll
                    for (int j = 0; j < Pr::N; ++j) {
                        const float2 dn0 = __ffma2_rn(g1[h].v[j], turn.s.v[j], __fmul2_rn(g0[h].v[j], turn.c.v[j]));
                        const float2 dn1 = __ffma2_rn(g1[h].v[j], turn.c.v[j], minus(__fmul2_rn(g0[h].v[j], turn.s.v[j])));
                        x0.v[j] = __fmul2_rn(x0.v[j], both(r));
                        x1.v[j] = __fmul2_rn(x1.v[j], both(r));
                        dw0.v[j] = __ffma2_rn(dn0, x0.v[j], dw0.v[j]);
                        dw1.v[j] = __ffma2_rn(dn1, x1.v[j], dw1.v[j]);
                        g0[h].v[j] = __fmul2_rn(dn0, w0.v[j]);
                        g1[h].v[j] = __fmul2_rn(dn1, w1.v[j]);
                        dot2 = __ffma2_rn(g0[h].v[j], x0.v[j], __ffma2_rn(g1[h].v[j], x1.v[j], dot2));
                    }
                    const float2 dot = both(-row_sum<L>(dot2.x + dot2.y) * (1.f / D));
#pragma unroll
                    for (int j = 0; j < Pr::N; ++j) {
                        g0[h].v[j] = __fmul2_rn(__ffma2_rn(x0.v[j], dot, g0[h].v[j]), both(r));
                        g1[h].v[j] = __fmul2_rn(__ffma2_rn(x1.v[j], dot, g1[h].v[j]), both(r));
                    }
                }
                if (live && h0 + hp + h < n_heads) {  // a padding row's gradient is zero
                    g0[h].store(dst + (hp + h) * D + e0);
                    g1[h].store(dst + (hp + h) * D + e1);
                }
            }
        }
    }
    depend_next();
    if (kind == 2) return;
#pragma unroll
    for (int j = 0; j < Pr::N; ++j) {
        part[slot][e0 + 2 * j] = dw0.v[j].x;
        part[slot][e0 + 2 * j + 1] = dw0.v[j].y;
        part[slot][e1 + 2 * j] = dw1.v[j].x;
        part[slot][e1 + 2 * j + 1] = dw1.v[j].y;
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kThreads) {
        float sum = 0.f;
#pragma unroll
        for (int sl = 0; sl < SLOTS; ++sl) sum += part[sl][d];
        a.partial[((long long)blockIdx.y * gridDim.x + blockIdx.x) * D + d] = sum;
    }
}

// dw of q (blockIdx.y = 0) and k (1): the partials of its head groups, in a fixed order, in
// 64 bits.  A CTA takes 8 dims with 32 threads each.
template <int D>
__global__ void __launch_bounds__(256) norm_rope_dw(const NormRopeArgs a, int grid_x) {
    __shared__ double part[8][8];
    const int kind = blockIdx.y, d = threadIdx.x % 8, slot = threadIdx.x / 8;
    const long long n = (long long)a.groups[kind] * grid_x;
    const float *p = a.partial + (kind ? (long long)a.groups[0] * grid_x * D : 0) + blockIdx.x * 8 + d;
    depend_wait();
    depend_next();
    double sum = 0.0;
#pragma unroll 8
    for (long long i = slot; i < n; i += 32) sum += (double)p[i * D];
    sum += __shfl_xor_sync(0xffffffffu, sum, 8);
    sum += __shfl_xor_sync(0xffffffffu, sum, 16);
    if (threadIdx.x % 32 < 8) part[threadIdx.x / 32][d] = sum;
    __syncthreads();
    if (threadIdx.x < 8) {
        sum = 0.0;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += part[i][d];
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
    // Four heads a thread from two CTAs an SM on.  us with one / four, bf16, 32 + 8 heads of 128:
    // 128 tokens 2.2 / 2.5, 384 (288 CTAs of four) 3.0 / 3.3, 512 (384) 3.4 / 3.4, 1,024 6.4 / 5.3,
    // 2,048 12.2 / 10.0; fp32, 12 + 4 heads of 64: 512 tokens (160) 2.2 / 2.2, 1,024 (320) 2.8 / 2.6,
    // 2,048 4.3 / 3.5.  With few heads the four loads are not all there: 4 + 1 heads of 128,
    // 2,048 tokens (384) 2.7 / 3.0.
    const bool longer = gx * (a.groups[0] + 2 * a.groups[1]) >= 2 * sm_count();
    if (!longer) set_groups(a, 1);
    return record_cuda(launch_dependent(longer ? norm_rope_kernel<T, D, kHeads> : norm_rope_kernel<T, D, 1>,
                                        dim3((unsigned)gx, a.groups[0] + 2 * a.groups[1]), kThreads, 0, 1, stream, a));
}

// CTAs along the tokens of the backward: one wave of 148 SMs over all head groups.  A
// fixed number, so that the workspace size needs no device.
long long bwd_grid_x(const hga_proj_t &p) {
    const int lanes = p.head_dim / (p.dtype == HGA_FP32 ? 8 : 16);
    const int slots = kThreads / lanes;
    const long long steps = ((long long)p.batch * p.seq_len + slots - 1) / slots;
    const int groups = (p.n_q_heads + kHeads - 1) / kHeads + 2 * ((p.n_kv_heads + kHeads - 1) / kHeads);
    const long long want = groups < 148 * kBwdCtas ? 148 * kBwdCtas / groups : 1;
    return steps < want ? steps : want;
}

template <typename T, int D> hga_status_t launch_bwd(NormRopeArgs a, long long gx, cudaStream_t stream) {
    set_groups(a, kHeads);
    const dim3 grid((unsigned)gx, a.groups[0] + 2 * a.groups[1]);
    const cudaError_t e = launch_dependent(norm_rope_bwd_kernel<T, D>, grid, kThreads, 0, 1, stream, a);
    if (e != cudaSuccess) return record_cuda(e);
    return record_cuda(launch_dependent(norm_rope_dw<D>, dim3(D / 8, 2), 256, 0, 1, stream, a, (int)gx));
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
