// Packing closed chunks into 4-bit records at detach time, and reading them back.
//
// "Long-Context Fine-Tuning with Limited VRAM", technical summary section 2.2:
// detached history is read, never differentiated, and its memory grows with the
// context; a 4-bit record (packed.cuh) is 72 D bytes against 256 D in bf16.
//
// Grid of a group with extremes mn, mx (K: a channel's 64 tokens, V: 64 channels of a
// token), c nearest to the value, ties to even:
//   s = bf16(fl(fl(mx - mn) fl(1 / 15))), 0 below 2^-100
//   z = bf16(fl(mn - 16 s)),   c = clamp(rne((x - z) / s) - 16, 0, 15), 0 where s = 0
// s and z are rounded first and the codes chosen for the rounded grid, so their
// rounding moves the grid and not the choice.  s = z = NaN when an element is not finite
// (the extremes propagate NaN, an infinity makes s infinite) or s or z is not: the
// group's values read as NaN.
//
// pack's floor is HBM: K and V are read once (the summaries come from the same read), and
// 0.28 of their bytes written.  One 256-thread CTA takes a chunk, all of its loads in
// flight; K's extremes and sums cross threads through shared memory, V's stay in the lanes
// of a row, and V's codes are turned there from token to channel order.  Choosing 16,384
// codes a chunk costs more issue time (0.68 of the slots) than its bytes cost bandwidth, so
// the choice is made of two-element FMAs and one multiply-add into the word.  1,792 bf16
// chunks of D = 128 packed and unpacked take 31.9 us (150 MB: 23 us at the measured copy
// rate); packed alone 20.5 us (75 MB: 11.5), in fp32 30.8 us (135 MB: 20.5).  Both took 65 us
// when each element took a rounding, a conversion and, near a border, a 64-bit decision, and
// 30.0 us without the marks of odd grids (below).  Four CTAs an SM (64 registers) against three
// gained 1.3 us; K and V in CTAs of their own took 41.5 us.
#include <cfloat>

#include "dependent.cuh"
#include "packed.cuh"

namespace hga {

namespace {

constexpr int kChunk = 64;
constexpr int kThreads = 256;

struct Grid {
    float s, z;
};

__device__ __forceinline__ float bf16_round(float x) { return __bfloat162float(__float2bfloat16_rn(x)); }

__device__ __forceinline__ Grid make_grid(float mn, float mx) {
    Grid g;
    g.s = bf16_round(__fmul_rn(__fsub_rn(mx, mn), 1.f / 15.f));
    if (g.s < 0x1p-100f) g.s = 0.f;
    g.z = bf16_round(fmaf(-16.f, g.s, mn));
    // fabsf(NaN) <= FLT_MAX is false
    if (!(fabsf(g.s) <= FLT_MAX) || !(fabsf(g.z) <= FLT_MAX)) g.s = g.z = __int_as_float(0x7FC00000);
    return g;
}

// s in the low and z in the high half of a word.
__device__ __forceinline__ uint32_t grid_bits(const Grid &g) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(g.s, g.z);
    return *reinterpret_cast<const uint32_t *>(&b);
}
__device__ __forceinline__ Grid grid_of(uint32_t b) {
    return {__uint_as_float(b << 16), __uint_as_float(b & 0xFFFF0000u)};
}

// 1 / (15 s) to within 2^-21, 0 for s = 0 (every element is code 0).
__device__ __forceinline__ float grid_inv(float s) { return s == 0.f ? 0.f : __fdividef(1.f / 15.f, s); }

// An element is decided again when it lies further than this many steps from the value of its
// approximated code (r of codes() below).  fp32 can tell, for most grids; in units of s, with
// s taken as 1 .. 2:
//   * (16 + c) s and borders have 14 significant bits, the last at 2^-8, and their sum with z is
//     exact for 2^-10 s <= |z| <= 2^14 s and for z = 0.  Grids of bf16 elements keep to that: a range is
//     no less than the last place of an extreme, and a z this small the difference of two
//     8-bit numbers.
//   * r is then rounded only if x is small beside s and a border lies next to x: fp32 elements
//     so near to a border, ties among them, count as further.  The only border as near to
//     a bf16 element without being equal to it (2^-14 s, twice what codes() rounds to a tie) is 0:
//     grids that have it are looked through for such elements (ties, 0.2% of Gaussian elements,
//     are too many to be decided again).
//   * x - z and 1 / (15 s) are normal numbers up to s = 2^120.
// odd_grid() names the others, and the bf16 grids with the border 0 (one Gaussian group in 600).
template <typename T> constexpr float kReach = sizeof(T) == 4 ? 0.5f - 0x1p-23f : 0.5f;
template <typename T> __device__ __forceinline__ bool odd_grid(const Grid &g, float inv) {
    if constexpr (sizeof(T) == 4) {
        const float z = fabsf(g.z);
        return g.s > 0x1p120f || (g.s != 0.f && (z > 0x1p14f * g.s || (z != 0.f && z < 0x1p-10f * g.s)));
    } else {
        const float m = rintf(fmaf(-15.f * inv, g.z, -0.5f)) + 0.5f;  // the border next to 0
        return g.s > 0x1p120f || (g.s != 0.f && fmaf(m, g.s, g.z) == 0.f);
    }
}
// While codes are chosen, the step of such a grid has its sign bit set: every r, meaningless
// then, is further than a negative number, without a comparison more on the common path.
constexpr uint32_t kOdd = 0x8000u;
// Whether an element of a grid with step s (as marked) is decided again, its r being further.
template <typename T> __device__ __forceinline__ bool again(float x, float s) {
    return sizeof(T) == 4 || !(s < 0.f) || s < -0x1p120f || (x != 0.f && fabsf(x) < -0x1p-14f * s);
}
template <typename T> __device__ __forceinline__ uint32_t mark_odd(uint32_t grid, float inv) {
    return odd_grid<T>(grid_of(grid), inv) ? grid | kOdd : grid;
}

__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Where the nibble of a word's element e starts, and of a staged byte.
template <bool kNibble> __device__ constexpr int code_shift(int e) {
    return kNibble ? 4 * (e >> 1) + 16 * (e & 1) : 8 * e;
}

// Codes of N elements in a word, approximated: p = (x - z) / (15 s) - 16/15 saturates to
// [0, 1] and 15 p is within 2^-17 of the quotient.  Rounding it to 2^-14 turns what lies that
// close to a border into a tie, which the rounding to an integer (adding 1.5 2^23 leaves the
// integer in the low bits) gives to the even code.  A true tie belongs there; an element
// that does not is more than half a step from its code, and r = x - ((16 + c) s + z) tells.
// r[e] is for the caller to compare with kReach s.
template <int N, bool kNibble>
__device__ __forceinline__ uint32_t codes(const float (&x)[N], const float (&ss)[N], const float (&zs)[N],
                                          const float (&inv)[N], float (&r)[N]) {
    constexpr float magic = 12582912.f, magic14 = 768.f;  // ulp 1 and 2^-14
    constexpr uint32_t magic_bits = 0x4B400000u;
    uint32_t w = 0, off = 0;
#pragma unroll
    for (int e = 0; e < N; e += 2) {
        const float2 y = __fadd2_rn(make_float2(x[e], x[e + 1]), make_float2(-zs[e], -zs[e + 1]));
        const float2 p = make_float2(__saturatef(fmaf(y.x, inv[e], -16.f / 15.f)),
                                     __saturatef(fmaf(y.y, inv[e + 1], -16.f / 15.f)));
        const float2 u = __ffma2_rn(p, make_float2(15.f, 15.f), make_float2(magic14, magic14));
        const float2 t = __fadd2_rn(u, make_float2(magic - magic14, magic - magic14));
        const float2 k = __fadd2_rn(t, make_float2(16.f - magic, 16.f - magic));
        const float2 g = __ffma2_rn(k, make_float2(-ss[e], -ss[e + 1]), make_float2(-zs[e], -zs[e + 1]));
        const float2 d = __fadd2_rn(make_float2(x[e], x[e + 1]), g);
        r[e] = d.x;
        r[e + 1] = d.y;
        // the constant bits of t add up to a constant, modulo 2^32
        w += __float_as_uint(t.x) * (1u << code_shift<kNibble>(e));
        w += __float_as_uint(t.y) * (1u << code_shift<kNibble>(e + 1));
        off += (magic_bits << code_shift<kNibble>(e)) + (magic_bits << code_shift<kNibble>(e + 1));
    }
    return w - off;
}

// A code, at most one off, decided by its borders (16 + k +- 1/2) s + z, which fp32 holds.
__device__ __forceinline__ uint32_t border_code(float x, const Grid &g, uint32_t k) {
    const float up = fmaf(16.5f + (float)k, g.s, g.z), dn = fmaf(15.5f + (float)k, g.s, g.z);
    const bool odd = k & 1;  // a tie leaves an odd code
    if (x > up || (x == up && odd))
        k = k < 15u ? k + 1u : k;
    else if (x < dn || (x == dn && odd))
        k = k > 0u ? k - 1u : k;
    // a NaN grid fails every comparison and keeps code 0; s = 0 has only code 0
    return g.s == 0.f ? 0u : k;
}

// The code of any grid with s > 0: x - z as the sum of its rounding y and what that lost, against
// the borders (q +- 1/2) s.  Rounding is monotonic, so y on one side of a border has x - z there
// too, and y on it leaves the decision to the rest.  Above s = 2^120 all three are scaled, so that
// x - z does not overflow.
__device__ __forceinline__ uint32_t exact_code(float x, const Grid &g) {
    const float f = g.s > 0x1p120f ? 0.0625f : 1.f, v = x * f, z = g.z * f, s = g.s * f;
    const float y = __fsub_rn(v, z), vr = __fadd_rn(y, z);
    const float rest = __fadd_rn(__fsub_rn(v, vr), __fsub_rn(__fsub_rn(vr, y), z));
    // within 2^-18 of the quotient: at most one border off
    int q = __float2int_rn(fminf(fmaxf(__fdividef(y, s), 16.f), 31.f));
    const float up = ((float)q + 0.5f) * s, dn = ((float)q - 0.5f) * s;
    const bool odd = q & 1;
    if (q < 31 && (y > up || (y == up && (odd ? rest >= 0.f : rest > 0.f))))
        ++q;
    else if (q > 16 && (y < dn || (y == dn && (odd ? rest <= 0.f : rest < 0.f))))
        --q;
    return (uint32_t)q - 16u;
}

__device__ __forceinline__ uint32_t decide(float x, uint32_t grid, uint32_t k) {
    const Grid g = grid_of(grid & ~kOdd);
    return grid & kOdd ? exact_code(x, g) : border_code(x, g, k);
}

// A word's codes decided again: four elements of one grid staged as bytes, or those of the 16
// bytes of elements (8 or 4) with a grid each that `which` names, as nibbles.  Few warps come
// here: one element in 2^15 of arbitrary ones, odd grids, and groups whose z lost more than half
// a step to its rounding; calls, so that the common path holds neither their code nor their
// registers (a call costs a warp 1 to 3 us).
__device__ __noinline__ uint32_t exact_bytes(float x0, float x1, float x2, float x3, uint32_t grid, uint32_t word) {
    return decide(x0, grid, word & 15u) | decide(x1, grid, word >> 8 & 15u) << 8 |
           decide(x2, grid, word >> 16 & 15u) << 16 | decide(x3, grid, word >> 24 & 15u) << 24;
}
template <typename T>
__device__ __noinline__ uint32_t exact_nibbles(uint4 x, const uint32_t *grids, uint32_t word, uint32_t which) {
    constexpr int N = Vec16<T>::N;
    const uint32_t raw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < N; ++e) {
        if (!(which >> e & 1u)) continue;
        const int sh = code_shift<true>(e);
        const uint32_t bf = raw[e / 2 % 4];  // bf16: the word that holds element e
        const float f = __uint_as_float(N == 4 ? raw[e % 4] : (e & 1 ? bf & 0xFFFF0000u : bf << 16));
        word = (word & ~(15u << sh)) | decide(f, grids[e], word >> sh & 15u) << sh;
    }
    return word;
}

// Extremes of elements, NaN if one is NaN.  For bf16 the word (-min, max) of a pair of
// halves, so that one instruction keeps both; for fp32 two floats.
template <typename T> struct Ext;
template <> struct Ext<__nv_bfloat16> {
    uint32_t w;
    __device__ __forceinline__ static uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    __device__ __forceinline__ static Ext row(const uint4 &u) {  // of 8 elements
        const uint32_t hi = max2(max2(u.x, u.y), max2(u.z, u.w));
        constexpr uint32_t sign = 0x80008000u;
        const uint32_t lo = max2(max2(u.x ^ sign, u.y ^ sign), max2(u.z ^ sign, u.w ^ sign));
        return {max2(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632))};
    }
    __device__ __forceinline__ Ext with(Ext o) const { return {max2(w, o.w)}; }
    __device__ __forceinline__ Ext shfl(int o) const { return {__shfl_xor_sync(0xffffffffu, w, o)}; }
    __device__ __forceinline__ float mn() const { return -__uint_as_float(w << 16); }
    __device__ __forceinline__ float mx() const { return __uint_as_float(w & 0xFFFF0000u); }
};
template <> struct Ext<float> {
    float lo, hi;
    __device__ __forceinline__ static Ext row(const uint4 &u) {  // of 4 elements
        const float x[4] = {__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w)};
        return {min_nan(min_nan(x[0], x[1]), min_nan(x[2], x[3])), max_nan(max_nan(x[0], x[1]), max_nan(x[2], x[3]))};
    }
    __device__ __forceinline__ Ext with(Ext o) const { return {min_nan(lo, o.lo), max_nan(hi, o.hi)}; }
    __device__ __forceinline__ Ext shfl(int o) const {
        return {__shfl_xor_sync(0xffffffffu, lo, o), __shfl_xor_sync(0xffffffffu, hi, o)};
    }
    __device__ __forceinline__ float mn() const { return lo; }
    __device__ __forceinline__ float mx() const { return hi; }
};

template <typename T> __device__ __forceinline__ uint32_t word_min(uint32_t a, uint32_t b) {  // lane-wise, NaN kept
    if constexpr (sizeof(T) == 2) {
        uint32_t r;
        asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    } else {
        return __float_as_uint(min_nan(__uint_as_float(a), __uint_as_float(b)));
    }
}
template <typename T> __device__ __forceinline__ uint32_t word_max(uint32_t a, uint32_t b) {
    if constexpr (sizeof(T) == 2)
        return Ext<__nv_bfloat16>::max2(a, b);
    else
        return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
}

// Thread (col, slot) owns VEC channels of the rows slot, slot + NSLOT, ...: the split of
// summaries_kernel, whose sums are repeated here in the same order bit for bit.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2)
    pack_kernel(const T *k, const T *v, long long head_stride, int n_chunks, int first_chunk, uint8_t *hist,
                long long cap, float *summ, long long summ_cap) {
    using P = Packed<D>;
    constexpr int VEC = Vec16<T>::N;
    constexpr int LPR = D / VEC;
    constexpr int NSLOT = kThreads / LPR;
    constexpr int ROWS = kChunk / NSLOT;
    constexpr int CS = D + 4;  // row stride of the staged V codes, bytes
    constexpr int WPR = D * (int)sizeof(T) / 4;  // words of a row
    __shared__ __align__(16) float part_sum[NSLOT][D + 4];
    __shared__ __align__(16) uint32_t part_mn[NSLOT][WPR + 4], part_mx[NSLOT][WPR + 4];
    __shared__ __align__(16) uint32_t kgrid[D];
    __shared__ __align__(16) float kinv[D];
    __shared__ __align__(16) uint8_t vcodes[kChunk * CS];
    const int tid = threadIdx.x;
    const long long slice = blockIdx.x / n_chunks;
    const int j = (int)(blockIdx.x % n_chunks);
    const int lane_col = tid % LPR, slot = tid / LPR;
    const int col = lane_col * VEC;
    const long long row0 = slice * head_stride + (long long)j * kChunk;
    uint8_t *rec = hist + (slice * cap + first_chunk + j) * P::kRecord;

    depend_wait();
    // the rows as they lie in memory; widened where they are used
    uint4 xr[ROWS], yr[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) xr[r] = *reinterpret_cast<const uint4 *>(k + (row0 + slot + r * NSLOT) * D + col);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) yr[r] = *reinterpret_cast<const uint4 *>(v + (row0 + slot + r * NSLOT) * D + col);
    auto widen = [](const uint4 &u, float (&f)[VEC]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (VEC == 8) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            } else {
                f[i] = __uint_as_float(w[i]);
            }
        }
    };

    // K: extremes and sum of every channel
    {
        float sum[VEC];
        uint4 mn = xr[0], mx = xr[0];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            float x[VEC];
            widen(xr[r], x);
#pragma unroll
            for (int e = 0; e < VEC; ++e) sum[e] = (r ? sum[e] : 0.f) + x[e];
            if (r) {
                mn = make_uint4(word_min<T>(mn.x, xr[r].x), word_min<T>(mn.y, xr[r].y), word_min<T>(mn.z, xr[r].z),
                                word_min<T>(mn.w, xr[r].w));
                mx = make_uint4(word_max<T>(mx.x, xr[r].x), word_max<T>(mx.y, xr[r].y), word_max<T>(mx.z, xr[r].z),
                                word_max<T>(mx.w, xr[r].w));
            }
        }
#pragma unroll
        for (int e = 0; e < VEC; e += 4)
            *reinterpret_cast<float4 *>(&part_sum[slot][col + e]) =
                make_float4(sum[e], sum[e + 1], sum[e + 2], sum[e + 3]);
        *reinterpret_cast<uint4 *>(&part_mn[slot][4 * lane_col]) = mn;
        *reinterpret_cast<uint4 *>(&part_mx[slot][4 * lane_col]) = mx;
    }

    // V: the extremes of every token and 64 channels lie in GL lanes.  Each exchange halves
    // the rows that a lane goes on with, until one is left; that lane makes the row's grid.
    constexpr int GL = 64 / VEC;  // lanes per group
    constexpr int PER = GL / ROWS;  // lanes that end up with the same row
    static_assert(PER >= 1, "a row's lanes outnumber the rows of a thread");
    uint32_t vgrid[ROWS];
    float vinv[ROWS];
    {
        Ext<T> ext[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) ext[r] = Ext<T>::row(yr[r]);
#pragma unroll
        for (int n = ROWS / 2; n >= 1; n /= 2) {
            const bool up = lane_col & (PER * n);
#pragma unroll
            for (int r = 0; r < n; ++r) {
                const Ext<T> give = up ? ext[r] : ext[r + n], keep = up ? ext[r + n] : ext[r];
                ext[r] = keep.with(give.shfl(PER * n));
            }
        }
#pragma unroll
        for (int o = PER / 2; o >= 1; o /= 2) ext[0] = ext[0].with(ext[0].shfl(o));
        const uint32_t bits = grid_bits(make_grid(ext[0].mn(), ext[0].mx()));
        const float own_inv = grid_inv(grid_of(bits).s);
        const int mine = (lane_col % GL) / PER;  // these lanes' row
        if (lane_col % PER == 0) {
            uint16_t *vs = reinterpret_cast<uint16_t *>(rec + P::kPart + P::kGridOff);
            const int at = (col / 64) * kChunk + slot + mine * NSLOT;
            vs[at] = (uint16_t)bits;
            vs[D + at] = (uint16_t)(bits >> 16);
        }
        const int lane0 = (tid & 31) & ~(GL - 1);
        const uint32_t marked = mark_odd<T>(bits, own_inv);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            vgrid[r] = __shfl_sync(0xffffffffu, marked, lane0 + PER * r);
            vinv[r] = __shfl_sync(0xffffffffu, own_inv, lane0 + PER * r);
        }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        float y[VEC];
        widen(yr[r], y);
        const Grid g = grid_of(vgrid[r]);
        float zs[VEC], iv[VEC], ss[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            zs[e] = g.z;
            iv[e] = vinv[r];
            ss[e] = g.s;
        }
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
            const float (&x4)[4] = reinterpret_cast<const float (&)[4]>(y[e]);
            const float (&s4)[4] = reinterpret_cast<const float (&)[4]>(ss[e]);
            const float (&z4)[4] = reinterpret_cast<const float (&)[4]>(zs[e]);
            const float (&i4)[4] = reinterpret_cast<const float (&)[4]>(iv[e]);
            float d[4];
            uint32_t w = codes<4, false>(x4, s4, z4, i4, d);
            if (fmaxf(fmaxf(fabsf(d[0]), fabsf(d[1])), fmaxf(fabsf(d[2]), fabsf(d[3]))) > kReach<T> * g.s &&
                (again<T>(x4[0], g.s) || again<T>(x4[1], g.s) || again<T>(x4[2], g.s) || again<T>(x4[3], g.s)))
                w = exact_bytes(x4[0], x4[1], x4[2], x4[3], vgrid[r], w);
            *reinterpret_cast<uint32_t *>(vcodes + (slot + r * NSLOT) * CS + col + e) = w;
        }
    }
    __syncthreads();
    if (tid < D) {
        float sum = 0.f;
#pragma unroll
        for (int s = 0; s < NSLOT; ++s) sum += part_sum[s][tid];
        if (summ) summ[(slice * summ_cap + first_chunk + j) * D + tid] = sum / (float)kChunk;
    } else if (tid < D + WPR) {
        const int w = tid - D;
        uint32_t mn = part_mn[0][w], mx = part_mx[0][w];
#pragma unroll
        for (int s = 1; s < NSLOT; ++s) {
            mn = word_min<T>(mn, part_mn[s][w]);
            mx = word_max<T>(mx, part_mx[s][w]);
        }
        uint16_t *gs = reinterpret_cast<uint16_t *>(rec + P::kGridOff);
        if constexpr (VEC == 8) {
            const uint32_t g0 = grid_bits(make_grid(__uint_as_float(mn << 16), __uint_as_float(mx << 16)));
            const uint32_t g1 =
                grid_bits(make_grid(__uint_as_float(mn & 0xFFFF0000u), __uint_as_float(mx & 0xFFFF0000u)));
            const float i0 = grid_inv(grid_of(g0).s), i1 = grid_inv(grid_of(g1).s);
            *reinterpret_cast<uint2 *>(&kgrid[2 * w]) = make_uint2(mark_odd<T>(g0, i0), mark_odd<T>(g1, i1));
            *reinterpret_cast<float2 *>(&kinv[2 * w]) = make_float2(i0, i1);
            *reinterpret_cast<uint32_t *>(gs + 2 * w) = __byte_perm(g0, g1, 0x5410);
            *reinterpret_cast<uint32_t *>(gs + D + 2 * w) = __byte_perm(g0, g1, 0x7632);
        } else {
            const uint32_t g = grid_bits(make_grid(__uint_as_float(mn), __uint_as_float(mx)));
            kinv[w] = grid_inv(grid_of(g).s);
            kgrid[w] = mark_odd<T>(g, kinv[w]);
            gs[w] = (uint16_t)g;
            gs[D + w] = (uint16_t)(g >> 16);
        }
    }

    depend_next();

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
    __syncthreads();

    // K codes: a word holds the channels of one thread (bf16) or of a lane pair (fp32)
    float ss[VEC], zs[VEC], iv[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const Grid g = grid_of(kgrid[col + e]);
        ss[e] = g.s;
        zs[e] = g.z;
        iv[e] = kinv[col + e];
    }
    uint32_t *kcodes = reinterpret_cast<uint32_t *>(rec);
    uint32_t kw[ROWS];
    float far[VEC];
#pragma unroll
    for (int r = 0; r < ROWS; r += 2) {  // two rows: their distances meet in a three-way maximum
        float x[VEC], d[2][VEC];
        widen(xr[r], x);
        kw[r] = codes<VEC, true>(x, ss, zs, iv, d[0]);
        widen(xr[r + 1], x);
        kw[r + 1] = codes<VEC, true>(x, ss, zs, iv, d[1]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) far[e] = fmaxf(fmaxf(r ? far[e] : 0.f, fabsf(d[0][e])), fabsf(d[1][e]));
    }
    bool redo = false;
#pragma unroll
    for (int e = 0; e < VEC; ++e) redo |= far[e] > kReach<T> * ss[e];
    if (redo) {
        uint32_t which = 0;
#pragma unroll
        for (int e = 0; e < VEC; ++e) which |= (far[e] > kReach<T> * ss[e] ? 1u : 0u) << e;
        if constexpr (sizeof(T) == 2) {
            uint32_t left = which;  // almost always one channel, and an odd one
#pragma unroll 1
            while (left) {
                const int e = __ffs(left) - 1;
                left &= left - 1u;
                const float s = grid_of(kgrid[col + e]).s;
                bool any = false;
#pragma unroll
                for (int r = 0; r < ROWS; ++r) {
                    const uint32_t w = e < 4 ? (e < 2 ? xr[r].x : xr[r].y) : (e < 6 ? xr[r].z : xr[r].w);
                    any |= again<T>(__uint_as_float(e & 1 ? w & 0xFFFF0000u : w << 16), s);
                }
                if (!any) which ^= 1u << e;
            }
        }
        if (which) {
#pragma unroll
            for (int r = 0; r < ROWS; ++r) kw[r] = exact_nibbles<T>(xr[r], &kgrid[col], kw[r], which);
        }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        uint32_t w = kw[r];
        if constexpr (VEC == 4) {  // elements 4 .. 7 of a word: pairs 2, 3
            w <<= 8 * (lane_col & 1);
            w |= __shfl_xor_sync(0xffffffffu, w, 1);
        }
        if (VEC == 8 || (lane_col & 1) == 0) kcodes[(slot + r * NSLOT) * (D / 8) + col / 8] = w;
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

// One CTA per record, bound by the bytes it writes (13.6 us for 1,792 bf16 chunks of
// D = 128, 75 MB: 11.5 at the copy rate; 33.0 us in fp32, 134 MB: 20.4).  K words are 8
// channels of a token, one 16-byte store (bf16) each; a V thread turns 8 channels x 8 tokens
// in registers.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) unpack_kernel(const uint8_t *hist, long long cap, int first_chunk,
                                                          int n_chunks, T *k, T *v, long long head_stride) {
    using P = Packed<D>;
    constexpr int OPR = D / 8;
    const int tid = threadIdx.x;
    const long long slice = blockIdx.x / n_chunks;
    const int j = (int)(blockIdx.x % n_chunks);
    const uint8_t *rec = hist + (slice * cap + first_chunk + j) * P::kRecord;
    const long long row0 = slice * head_stride + (long long)j * kChunk;
    depend_wait();
    depend_next();
    if (tid < kThreads / 2) {
        const int o = tid % OPR;
        uint32_t s[4], z[4], r[4];
        load4(rec + P::kGridOff + 16 * o, s);
        load4(rec + P::kGridOff + P::kGridHalf + 16 * o, z);
        // a load may not pass a store: four words at once (all eight of D = 128: 35.5 us for
        // 1,792 fp32 chunks against 33.0)
        constexpr int STEP = kThreads / 2 / OPR, AT_ONCE = 4;
#pragma unroll
        for (int row = 0; row < kChunk; row += AT_ONCE * STEP) {
            uint32_t w[AT_ONCE];
#pragma unroll
            for (int u = 0; u < AT_ONCE; ++u)
                w[u] = reinterpret_cast<const uint32_t *>(rec)[(row + u * STEP + tid / OPR) * OPR + o];
#pragma unroll
            for (int u = 0; u < AT_ONCE; ++u) {
                packed_octet(w[u], s, z, r);
                store8(k + (row0 + row + u * STEP + tid / OPR) * D + 8 * o, r);
            }
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
    return record_cuda(launch_dependent(pack_kernel<T, D>, (unsigned)(slices * n_chunks), kThreads, 0, 1, stream,
                                        static_cast<const T *>(k), static_cast<const T *>(v), head_stride, n_chunks,
                                        first_chunk, hist, cap, summ, summ_cap));
}

template <typename T, int D>
hga_status_t unpack_t(const uint8_t *hist, int cap, long long slices, int first_chunk, int n_chunks, void *k, void *v,
                      long long head_stride, cudaStream_t stream) {
    return record_cuda(launch_dependent(unpack_kernel<T, D>, (unsigned)(slices * n_chunks), kThreads, 0, 1, stream,
                                        hist, cap, first_chunk, n_chunks, static_cast<T *>(k), static_cast<T *>(v),
                                        head_stride));
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
