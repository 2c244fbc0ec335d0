// fa_cache_kernel.cuh -- the 4-bit key/value cache: append, read, attention
// against it and the weights of its tokens, for GB300 (sm_103a).
//
// Format.  A cache holds, for K and for V, codes [B, Hkv, C, D/2] (two 4-bit
// codes to a byte, the even channel in the low half) and params [B, Hkv, C, 2]
// in the cache's 16-bit type: a row x of D values has
//   min = min_d x_d,  scale = t((max_d x_d - min) / 15),
//   code_d = clamp(round_half_even((x_d - min) / scale), 0, 15)  (0 if scale = 0)
// and stands for min + code_d * scale.  min is an element of the row, so it is
// held exactly; the codes are chosen for the scale as it is held.
//
// Attention.  Query row (g, i) of a key head -- query head h Hkv-group member
// g, the i-th of the Nq last tokens of a sequence of len tokens -- sits at
// position p = len - Nq + i and sees tokens j <= p with j >= p - left (left <
// 0: no bound) or j < sinks:
//   x_j = scale * (ks_j sum_d u_jd q_d + kmin_j sum_d q_d),  p_j = exp(x_j - m)
//   O = sum_j (p_j vs_j) u'_j + sum_j p_j vmin_j  over  sum_j p_j
// with u, u' the integer codes: scale and minimum stay outside the products,
// so the matrix instructions see small integers (exact in 16 bits) against q
// (exact, the input) and against w_j = p_j vs_j (rounded to 16 bits).
//
// What bounds it: a decoded token reads every visible row once, D/2 + 4 bytes
// for each of K and V, and does 4 G Nq D operations on it -- HBM, at the few
// query rows per key head of decoding, if unpacking keeps up: 16 tokens are 64
// codes per lane for each of K and V, about five integer operations per eight.
// Hence mma.sync and not tcgen05 at those: the codes go from shared memory
// through registers (unpacking) straight into A fragments (16 tokens or channels
// x 16) with the 8 query rows as the N dimension, where tcgen05 would want the
// unpacked operand written back to shared memory or TMEM first, and its M =
// 128 rows are 16 times what a decode step has.
// More rows per key head (drafted tokens, the end of a prompt) come in blocks
// of 16, each of which reads and unpacks the key head's rows again, so the time
// grows with them: 16 sequences of 16001 to 32768 tokens, 8 key heads, D = 128,
// 8 / 16 / 32 / 64 rows: 79 / 108 / 196 / 376 us, where the bytes take 63 at
// each.  One pass for all rows would be a product for tcgen05, as the weights
// have it (fa_cache_rows.cu); the attention has none.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace fa {
namespace cache {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnit = 64;      // tokens per unit of work handed to the CTAs
constexpr int kSub = 32;       // tokens a warp takes at a time
constexpr int kStages = 3;     // kSub-token stages per warp, two of them in flight
constexpr int kMinUnits = 4;   // units per CTA, at least: half a round of the CTA's eight warps
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eRest = 1.9259629911266175e-8f;   // log2(e) - kLog2e
constexpr float kLn2f = 0.69314718055994530942f;
// The reference maximum m of a query row moves only when a score exceeds it
// by more than kSlack (log2 units): p stays below 2^kSlack, far inside fp32's
// range, and the sums are divided by one another at the end, so no precision
// is lost; most steps then take one vote instead of a reduction and a rescale.
constexpr float kSlack = 8.f;

struct Params {
    const uint8_t *kc;        // K codes [B, Hkv, C, D/2]
    const uint32_t *kp;       // K params [B, Hkv, C]: scale (low half), minimum
    const uint8_t *vc;        // V codes, params
    const uint32_t *vp;
    const void *q;            // [B, H, Nq, D]
    void *o;                  // [B, H, Nq, D]
    float *lse;               // [B, H, Nq]: written (attention) or read (weights)
    float *acc;               // weights: [B, Hkv, C]
    const int *lens;          // [B]
    int B, Hkv, C;
    int rows;                 // query rows per key head: (H / Hkv) * Nq
    int Nq;
    int RB;                   // row blocks per key head (tiles of 8 NT rows); weights: 1
    int whole;                // attention: no tile is cut (short caches)
    int left, sinks;          // left < 0: no window
    int accumulate;           // weights: add to acc instead of writing it
    float qk2;                // scale * log2(e)
    float *part_o;            // attention: [2 * grid slots][8 NT][D], not yet divided by l
    float2 *part_ml;          // [2 * grid slots][8 NT]
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void launch_dependents()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ void grid_wait()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// 16 or 4 bytes global -> shared, asynchronously; `real` false writes zeros
// and reads nothing.
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool real)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}

__device__ __forceinline__ void cp4(uint32_t dst, const void *src, bool real)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(real ? 4 : 0) : "memory");
}

__device__ __forceinline__ void cp_commit()
{
    asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// D[16 x 8] += A[16 x 16] B[16 x 8], fp16 operands, fp32 accumulation.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of 16-bit values held row-wise by the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Codes as fp16 operands: a code left in place in the low byte of a half is
// the subnormal code * 2^-24 (bits 0..3) or 16 code * 2^-24 (bits 4..7), exact.
// So one logic operation unpacks two codes, and a word of eight takes one
// shift besides -- the integer pipe, at half the rate of the others, is what
// unpacking is bound by.  The attention's go to the tensor core like that,
// the factor 16 taken out of the other operand or the result.  The weights,
// an fp32 result, bring K's to (code - 7.5) 2^-9 by one packed multiply-add
// more, exact again: the tensor core aligns a subnormal's product by its
// nominal exponent, which cuts low bits off the sum, and codes centred at
// their middle keep the sums as small as the scores (a weight's error against
// float64: 2.8e-7 with it, 1.1e-6 without).
constexpr uint32_t kEven = 0x000F000Fu, kOdd = 0x00F000F0u;
constexpr float kCodeUnit = 16777216.f;   // 2^24

__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

__device__ __forceinline__ uint32_t centred_even(uint32_t w)
{
    return hfma2(w & kEven, 0x78007800u, 0xA380A380u);   // * 2^15 - 7.5 * 2^-9
}

__device__ __forceinline__ uint32_t centred_odd(uint32_t w)
{
    return hfma2(w & kOdd, 0x68006800u, 0xA380A380u);    // * 2^11 - 7.5 * 2^-9
}

template <bool BF16>
__device__ __forceinline__ float to_float(uint32_t half16)
{
    return BF16 ? __uint_as_float(half16 << 16) : __half2float(__ushort_as_half((unsigned short)half16));
}

template <bool BF16>
__device__ __forceinline__ uint32_t from_float(float x)
{
    return BF16 ? (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(x)) : (uint32_t)__half_as_ushort(__float2half_rn(x));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float exp2i(int e)
{
    return __int_as_float((e + 127) << 23);
}

// ------------------------------------------------------------------ append, read

// What one row's codes are computed from, multiplied by `k`, a power of two
// that keeps differences, scale and reciprocal inside fp32's normal range (1
// but for extreme rows).
struct RowScale {
    float mn, sc, inv, k;
    uint32_t params;   // as held: scale, minimum
    bool flat;         // scale 0, or a row that is not finite: codes 0
    bool exact;        // x - mn or the quotient may need more than fp32: code_of for every value
};

template <bool BF16>
__device__ __forceinline__ RowScale row_scale(float mn, float mx)
{
    RowScale r;
    r.k = 1.f;
    r.exact = false;
    if (!(fabsf(mn) < INFINITY && fabsf(mx) < INFINITY)) {   // an infinity or NaN in the row: it stands for NaN
        r.params = BF16 ? 0x7FC07FC0u : 0x7E007E00u;
        r.flat = true;
        r.mn = r.sc = r.inv = 0.f;
        return r;
    }
    float range = mx - mn;
    if (BF16) {
        if (range > 3.0e38f)   // the range overflows: in quarters
            r.k = 0.25f;
        else if (range > 0.f && range < 8.0e-25f)
            r.k = 1.2089258196146292e24f;   // 2^80
        if (r.k != 1.f)
            range = mx * r.k - mn * r.k;
    }
    float sc = __fdiv_rn(range, 15.f);
    if (BF16 && r.k != 1.f)
        sc = __fdiv_rn(sc, r.k);   // (exact but for a scale that ends subnormal)
    r.params = from_float<BF16>(sc);
    const float held = to_float<BF16>(r.params);
    r.params |= from_float<BF16>(mn) << 16;
    r.flat = held == 0.f;
    r.sc = held * r.k;
    r.mn = mn * r.k;
    r.inv = __frcp_rn(r.sc);
    // a scale so much smaller than range / 15 that codes pass 15, or a
    // minimum so small that x - mn rounds
    r.exact = range * r.inv > 15.49f || (mn != 0.f && fabsf(mn) < fabsf(mx) * (BF16 ? 0x1p-15f : 0x1p-12f));
    return r;
}

// round_half_even((x - mn) / sc) clamped to 0..15, exactly: the quotient by the
// reciprocal, then the residual a - (q -+ 1/2) sc decides next to a border,
// with the rounding error of a = x - mn added back.
static __device__ __noinline__ uint32_t code_of(float x, float mn, float sc, float inv)
{
    const float a = x - mn;
    const float bb = a - x;
    const float e = (x - (a - bb)) + (-mn - bb);
    float q = fminf(rintf(a * inv), 16.f);
    const float t = fmaf(-q, sc, a);
    const float over = (t - 0.5f * sc) + e, under = (t + 0.5f * sc) + e;
    if (over > 0.f || (over == 0.f && ((int)q & 1)))
        q += 1.f;
    else if (under < 0.f || (under == 0.f && ((int)q & 1)))
        q -= 1.f;
    return (uint32_t)fminf(fmaxf(q, 0.f), 15.f);
}

// The codes of eight values.  Where x - mn is exact (fp16: magnitudes within
// 2^12 of one another, bf16: 2^15: `exact` false), the quotient a / sc
// corrected once by its residual -- the final step of Markstein's division --
// is a half-integer only if the true one is, so that rounding it half to even
// by adding and taking off 1.5 * 2^23 gives the code.  (Such values are not
// rare: 16-bit values over a 16-bit scale hit a border about once in 300.)
// Four codes at a time are summed as code * 16^i in one float, exact in 16
// bits.  With `exact`, values next to a border are decided by code_of.
__device__ __forceinline__ uint32_t codes_of(const float (&x)[8], const RowScale &r, bool exact)
{
    constexpr float kRound = 12582912.f;
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = x[i] - r.mn, f0 = a * r.inv;
        const float f = fmaf(fmaf(-f0, r.sc, a), r.inv, f0);
        s[i / 4] = fmaf((f + kRound) - kRound, (float)(1 << (4 * (i % 4))), s[i / 4]);
    }
    uint32_t w = (uint32_t)s[0] | ((uint32_t)s[1] << 16);
    if (exact) {
        float far = 0.f, top = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float f = (x[i] - r.mn) * r.inv;
            far = fmaxf(far, fabsf(f - ((f + kRound) - kRound)));
            top = fmaxf(top, f);
        }
        if (far > 0.4999f || top > 15.49f) {
            w = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w |= code_of(x[i], r.mn, r.sc, r.inv) << (4 * i);
        }
    }
    return w;
}

// Position of new token i of sequence b in the cache, or -1: not counted in,
// or outside [0, C).
__device__ __forceinline__ int slot_of(const int *start, const int *count, int b, int i, int N, int C)
{
    const int n = count ? count[b] : N;
    const long long at = (long long)start[b] + i;
    return (i < n && at >= 0 && at < C) ? (int)at : -1;
}

// Minima of two packed 16-bit values each; a NaN wins.
template <bool BF16>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b)
{
    uint32_t d;
    if (BF16)
        asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else
        asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

template <bool BF16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
{
    uint32_t d;
    if (BF16)
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// A row's 16 channels of this lane: minimum and maximum over the row's lanes
// (the pair (min, -max) goes through the shuffles as one word), codes, stores.
template <int D, bool BF16>
__device__ __forceinline__ void append_row(const uint4 (&x4)[2], int part, uint32_t group, uint8_t *codes, uint32_t *params)
{
    const uint32_t xw[8] = {x4[0].x, x4[0].y, x4[0].z, x4[0].w, x4[1].x, x4[1].y, x4[1].z, x4[1].w};
    uint32_t lo = xw[0], hi = xw[0], small = xw[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo = min2<BF16>(lo, xw[i]);
        hi = max2<BF16>(hi, xw[i]);
        small = min2<BF16>(small, xw[i] & 0x7FFF7FFFu);
    }
    uint32_t both = min2<BF16>(__byte_perm(lo, hi ^ 0x80008000u, 0x5410), __byte_perm(lo, hi ^ 0x80008000u, 0x7632));
#pragma unroll
    for (int m = D / 32; m > 0; m /= 2)
        both = min2<BF16>(both, __shfl_xor_sync(group, both, m));
    const RowScale r = row_scale<BF16>(to_float<BF16>(both & 0xffffu), -to_float<BF16>(both >> 16));
    uint2 w = make_uint2(0u, 0u);
    if (!r.flat) {
        float x[2][8];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            x[i / 8][i % 8] = to_float<BF16>((i & 1) ? xw[i / 2] >> 16 : xw[i / 2] & 0xffffu);
        if (r.k != 1.f) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                x[i / 8][i % 8] *= r.k;
        }
        // a value far smaller than the minimum's magnitude: x - mn may round
        const float least = fminf(to_float<BF16>(small & 0xffffu), to_float<BF16>(small >> 16));
        const bool exact = r.exact || least * r.k < fabsf(r.mn) * (BF16 ? 0x1p-15f : 0x1p-12f);
        w = make_uint2(codes_of(x[0], r, exact), codes_of(x[1], r, exact));
    }
    *reinterpret_cast<uint2 *>(codes + part * 8) = w;
    if (part == 0)
        *params = r.params;
}

// One group of D / 16 lanes per new token and head, K and V both (four loads
// in flight per lane), 16 channels a lane: the row's minimum, scale and
// reciprocal are shared by as many codes.  It reads 2 x 2 D bytes and writes
// 2 x (D/2 + 4) per token and head, at about a dozen instructions a value.
template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads)
    append_kernel(const uint16_t *kn, const uint16_t *vn, uint8_t *kc, uint32_t *kp, uint8_t *vc, uint32_t *vp,
                  const int *start, const int *count, int Hkv, int N, int C, uint32_t rows)
{
    constexpr int kTpr = D / 16;
    const uint32_t row = blockIdx.x * (kThreads / kTpr) + threadIdx.x / kTpr;   // (below 2^31 + a block's rows)
    if (row >= rows)   // whole groups leave together
        return;
    const int part = threadIdx.x % kTpr;
    const uint4 *ks = reinterpret_cast<const uint4 *>(kn + (size_t)row * D) + 2 * part;
    const uint4 *vs = reinterpret_cast<const uint4 *>(vn + (size_t)row * D) + 2 * part;
    const uint4 k4[2] = {__ldg(ks), __ldg(ks + 1)}, v4[2] = {__ldg(vs), __ldg(vs + 1)};
    const uint32_t bh = row / (uint32_t)N;
    const int i = (int)(row - bh * N);
    const int at = slot_of(start, count, (int)(bh / (uint32_t)Hkv), i, N, C);
    if (at < 0)
        return;
    const int lane = threadIdx.x % 32;
    const uint32_t group = ((1u << kTpr) - 1u) << (lane & ~(kTpr - 1));
    const size_t dst = (size_t)bh * C + at;
    append_row<D, BF16>(k4, part, group, kc + dst * (D / 2), kp + dst);
    append_row<D, BF16>(v4, part, group, vc + dst * (D / 2), vp + dst);
}

template <bool BF16>
__device__ __forceinline__ uint4 values_of(uint32_t w, uint32_t params)
{
    const float sc = to_float<BF16>(params & 0xffffu), mn = to_float<BF16>(params >> 16);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // (the code as the low bits of 2^23, taken off again: no conversion instruction)
        const float a = __uint_as_float(((w >> (8 * i)) & 15u) | 0x4B000000u) - 8388608.f;
        const float b = __uint_as_float(((w >> (8 * i + 4)) & 15u) | 0x4B000000u) - 8388608.f;
        const float lo = fmaf(a, sc, mn), hi = fmaf(b, sc, mn);
        o[i] = from_float<BF16>(lo) | (from_float<BF16>(hi) << 16);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// The values that rows start[b] .. start[b] + N - 1 stand for, rounded once
// to the cache's type; rows not counted in or outside the cache are zeros.
template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads)
    read_kernel(const uint8_t *kc, const uint32_t *kp, const uint8_t *vc, const uint32_t *vp, uint16_t *ko, uint16_t *vo,
                const int *start, const int *count, int Hkv, int N, int C, uint32_t rows)
{
    constexpr int kTpr = D / 8;
    const uint32_t row = blockIdx.x * (kThreads / kTpr) + threadIdx.x / kTpr;
    if (row >= rows)
        return;
    const int part = threadIdx.x % kTpr;
    const uint32_t bh = row / (uint32_t)N;
    const int i = (int)(row - bh * N);
    const int at = slot_of(start, count, (int)(bh / (uint32_t)Hkv), i, N, C);
    uint4 k4 = make_uint4(0u, 0u, 0u, 0u), v4 = k4;
    if (at >= 0) {
        const size_t src = (size_t)bh * C + at;
        const uint32_t kw = *reinterpret_cast<const uint32_t *>(kc + src * (D / 2) + part * 4);
        const uint32_t vw = *reinterpret_cast<const uint32_t *>(vc + src * (D / 2) + part * 4);
        k4 = values_of<BF16>(kw, kp[src]);
        v4 = values_of<BF16>(vw, vp[src]);
    }
    reinterpret_cast<uint4 *>(ko + (size_t)row * D)[part] = k4;
    reinterpret_cast<uint4 *>(vo + (size_t)row * D)[part] = v4;
}

// ------------------------------------------------------------------ work decomposition

// The units (kUnit tokens) that a sequence's visible tokens lie in: the sinks'
// [0, su), then [ks, ks + n - su); every sequence has at least one, so that
// rows which see nothing get their O = 0 and LSE = -inf written.
struct Span {
    int len;   // clamped to [0, C]
    int su, ks, n;
    __device__ int token(int u) const { return (u < su ? u : u - su + ks) * kUnit; }
};

__device__ __forceinline__ Span span_of(const Params &p, int b)
{
    Span s;
    int len = p.lens[b];
    s.len = len = len < 0 ? 0 : (len > p.C ? p.C : len);
    const int ke = (len + kUnit - 1) / kUnit;
    s.su = 0;
    s.ks = 0;
    if (p.left >= 0) {
        const long long lo = (long long)len - p.Nq - p.left;   // the first query's first token in the window
        if (lo > 0) {
            s.su = ((p.sinks < len ? p.sinks : len) + kUnit - 1) / kUnit;
            s.ks = (int)(lo / kUnit);
            s.ks = s.ks < s.su ? s.su : s.ks;
        }
    }
    s.n = s.su + ke - s.ks;
    s.n = s.n < 1 ? 1 : s.n;
    return s;
}

// CTAs that take part of `grid`: each has at least kMinUnits units.
__device__ __forceinline__ long long parts_of(long long total, int grid)
{
    const long long g = total / kMinUnits;
    return g < 1 ? 1 : (g < grid ? g : grid);
}

// Where the share of CTA k of `grid` begins.  Tiles are ordered by sequence,
// key head and row block; a tile of sequence b is span_of(b).n units, and of
// the U units in all, CTA k of the G that take part has [U k / G, U (k + 1) / G).
struct Where {
    long long total, parts;   // U, G
    long long first;          // U k / G (0 for k >= G)
    long long before;         // units of the sequences before b
    int b;                    // the sequence that holds unit `first`
};

// U k / G for k <= G (in 32 bits where it fits: a 64-bit division is some
// hundred instructions).
__device__ __forceinline__ long long share_of(const Where &w, int k)
{
    if (w.total < (1ll << 22))   // (k is below 2^10)
        return (uint32_t)w.total * (uint32_t)k / (uint32_t)w.parts;
    return w.total * k / w.parts;
}

// Tile (key head and row block) of its sequence, of `n` units a tile, that holds
// unit d of the sequence's.
__device__ __forceinline__ int tile_of(long long d, int n)
{
    return d < (1ll << 31) ? (int)((uint32_t)d / (uint32_t)n) : (int)(d / n);
}

// Called by every thread of the block, kThreads or more (it reads all of lens);
// `scratch` holds kWarps + 2 values.  The first kThreads threads take
// consecutive sequences; an exclusive scan over the threads' sums, then the
// owning thread walks its own.
__device__ inline Where locate(const Params &p, int k, int grid, long long *scratch)
{
    const int t = threadIdx.x, lane = t % 32, warp = t / 32;
    const int per = (p.B + kThreads - 1) / kThreads;
    const long long HR = (long long)p.Hkv * p.RB;
    long long sum = 0;
    if (t < kThreads)
        for (int i = t * per; i < (t + 1) * per && i < p.B; ++i)
            sum += span_of(p, i).n * HR;
    long long inc = sum;
#pragma unroll
    for (int m = 1; m < 32; m *= 2) {
        const long long v = __shfl_up_sync(0xffffffffu, inc, m);
        if (lane >= m)
            inc += v;
    }
    if (lane == 31 && warp < kWarps)
        scratch[warp] = inc;
    __syncthreads();
    Where w{0, 0, 0, 0, 0};
    long long before = inc - sum;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        before += i < warp ? scratch[i] : 0;
        w.total += scratch[i];
    }
    w.parts = parts_of(w.total, grid);
    w.first = k < w.parts ? w.total * k / w.parts : 0;
    if (w.first >= before && w.first < before + sum) {
        int b = t * per;
        for (;; ++b) {
            const long long n = span_of(p, b).n * HR;
            if (w.first < before + n)
                break;
            before += n;
        }
        scratch[kWarps] = before;
        scratch[kWarps + 1] = b;
    }
    __syncthreads();
    w.before = scratch[kWarps];
    w.b = (int)scratch[kWarps + 1];
    return w;
}

// The same, quicker where a warp can hold a sequence to a lane: every warp for
// itself, without the barriers (the weights, 8 sequences: 17.4 -> 17.1 us, 64
// rows 24.6 -> 23.7).  Not for the attention, whose registers are full: it
// spilled 116 bytes and took 80.4 us for 78.2.
__device__ inline Where locate_quick(const Params &p, int k, int grid, long long *scratch)
{
    if (p.B > 32)
        return locate(p, k, grid, scratch);
    const int lane = threadIdx.x % 32;
    const long long sum = lane < p.B ? span_of(p, lane).n * ((long long)p.Hkv * p.RB) : 0;
    long long inc = sum;
#pragma unroll
    for (int m = 1; m < 32; m *= 2) {
        const long long v = __shfl_up_sync(0xffffffffu, inc, m);
        if (lane >= m)
            inc += v;
    }
    Where w;
    w.total = __shfl_sync(0xffffffffu, inc, 31);
    w.parts = parts_of(w.total, grid);
    w.first = k < w.parts ? share_of(w, k) : 0;
    w.b = __ffs(__ballot_sync(0xffffffffu, w.first < inc)) - 1;   // (inc never falls, and ends above `first`)
    w.before = __shfl_sync(0xffffffffu, inc - sum, w.b);
    return w;
}

// ------------------------------------------------------------------ attention

template <int D>
struct Layout {
    static constexpr int kRow = D / 2;                     // bytes of codes per token
    static constexpr int kCodes = kSub * kRow;             // per stage, K or V
    static constexpr int kStage = 2 * kCodes + 2 * kSub * 4;
    static constexpr int kKeyStage = kCodes + kSub * 4;    // weights: K alone
    static constexpr int kWords = D / 32;                  // words of 8 codes per lane and K row
    static constexpr int kVWords = D / 64;                 // words per lane and V row
    static constexpr int kMTiles = D / 16;                 // 16-channel tiles of O^T
};

// Shared-memory offset of 16-byte chunk j of V row t within its stage.  The
// lanes of a warp read, for c = 0..3, tokens 2c (or 2c + 1) of a block of
// eight; rows are placed, and at D = 128 their halves swapped, so that those
// four rows fall into different banks.
template <int D>
__device__ __forceinline__ uint32_t v_chunk(int t, int j)
{
    const int block = t >> 3, k = (t >> 1) & 3, e = t & 1;
    if (D == 128)
        return (uint32_t)(block * 512 + ((k >> 1) * 4 + e * 2 + (k & 1)) * 64 + ((j ^ ((k >> 1) * 2)) * 16));
    return (uint32_t)(block * 256 + (e * 4 + k) * 32 + j * 16);
}

// One key head's rows, this lane's first bytes of a step at token 0.
template <int D>
struct Rows {
    const uint8_t *kc, *vc;
    const uint32_t *kp, *vp;

    __device__ Rows(const Params &p, long long bh)
    {
        const int lane = threadIdx.x % 32;
        const long long row = bh * p.C;
        kc = p.kc + row * Layout<D>::kRow + lane * 16;
        vc = p.vc + row * Layout<D>::kRow + lane * 16;
        kp = p.kp + row + lane;
        vp = p.vp + row + lane;
    }
};

// Issue the loads of tokens t0 .. t0 + 31 into a stage (V left out for the
// weights); tokens from `len` on are zeros.  Always commits a group.
template <int D, bool VALUES>
__device__ __forceinline__ void load_stage(const Rows<D> &rows, uint32_t stage, int t0, int len, bool any)
{
    using L = Layout<D>;
    const int lane = threadIdx.x % 32;
    constexpr int kPer = L::kRow / 16;   // 16-byte chunks per row; 32 lanes hold 512 bytes of consecutive rows
    if (any) {
        const uint8_t *kc = rows.kc + (long long)t0 * L::kRow, *vc = rows.vc + (long long)t0 * L::kRow;
        const uint32_t dk = stage + lane * 16, dv = stage + L::kCodes + v_chunk<D>(lane / kPer, lane % kPer);
        const uint32_t par = stage + (VALUES ? 2 : 1) * L::kCodes + lane * 4;
        if (t0 + kSub <= len) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {   // (v_chunk moves by 512 bytes per 512 bytes of rows)
                cp16(dk + i * 512, kc + i * 512, true);
                if (VALUES)
                    cp16(dv + i * 512, vc + i * 512, true);
            }
            cp4(par, rows.kp + t0, true);
            if (VALUES)
                cp4(par + kSub * 4, rows.vp + t0, true);
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const bool real = t0 + lane / kPer + i * (32 / kPer) < len;
                cp16(dk + i * 512, real ? kc + i * 512 : rows.kc, real);
                if (VALUES)
                    cp16(dv + i * 512, real ? vc + i * 512 : rows.vc, real);
            }
            const bool real = t0 + lane < len;
            cp4(par, real ? rows.kp + t0 : rows.kp, real);
            if (VALUES)
                cp4(par + kSub * 4, real ? rows.vp + t0 : rows.vp, real);
        }
    }
    cp_commit();
}

__device__ __forceinline__ uint32_t lds32(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

// The query rows as B fragments (16 channels x 8 rows each), in the channel
// order in which K's codes come out of their words: lane (r = lane / 4, c =
// lane % 4) holds row 8 nt + r, channels [c D/4, (c + 1) D/4); word w of them
// gives two fragments, (0, 4 | 1, 5) and (2, 6 | 3, 7), the odd channels
// divided by 16 where K's codes are taken as they are (not CENTRED).  As fp16: a row is multiplied by the power of two that brings
// its largest element to [2^14, 2^15), so a bf16 or fp16 element is exact
// unless it is 2^-24 of the largest or less, and then off by 2^-40 of it.
// `mul` takes the power, the codes' unit and the softmax scale (log2 units)
// out again; `sum` is sum_d q_d in those units; both for the two rows
// (columns of S^T) of this lane.
template <int D, bool BF16, int NT, bool CENTRED>
struct Queries {
    using L = Layout<D>;
    uint32_t f[NT][L::kWords * 2][2];
    float sum[NT][2], mul[NT][2];

    __device__ void load(const Params &p, long long row0, int nrows)
    {
        const int lane = threadIdx.x % 32, r = lane / 4, c = lane % 4;
        const uint32_t *q = reinterpret_cast<const uint32_t *>(p.q);   // channel pairs
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int n = 8 * nt + r;
            float x[L::kWords][8];
            float s = 0.f, mx = 0.f;
#pragma unroll
            for (int w = 0; w < L::kWords; ++w) {
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (n < nrows)
                    v = __ldg(reinterpret_cast<const uint4 *>(q + (row0 + n) * (D / 2) + (c * L::kWords + w) * 4));
                const uint32_t xw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[w][i] = to_float<BF16>((i & 1) ? xw[i / 2] >> 16 : xw[i / 2] & 0xffffu);
                    s += x[w][i];
                    mx = fmaxf(mx, fabsf(x[w][i]));
                }
            }
#pragma unroll
            for (int m = 1; m < 4; m *= 2) {
                s += __shfl_xor_sync(0xffffffffu, s, m);
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, m));
            }
            // (queries of 2^114 and more overflow fp16, and their rows end as NaN)
            int e = mx > 0.f ? 14 - (int)((__float_as_uint(mx) >> 23) & 255u) + 127 : 0;
            e = e > 100 ? 100 : (e < -100 ? -100 : e);
            const float up = exp2i(e), up1 = CENTRED ? up : up * 0.0625f;
#pragma unroll
            for (int w = 0; w < L::kWords; ++w) {
                f[nt][2 * w][0] = pack_f16(x[w][0] * up, x[w][4] * up);
                f[nt][2 * w][1] = pack_f16(x[w][1] * up1, x[w][5] * up1);
                f[nt][2 * w + 1][0] = pack_f16(x[w][2] * up, x[w][6] * up);
                f[nt][2 * w + 1][1] = pack_f16(x[w][3] * up1, x[w][7] * up1);
            }
            const float back = p.qk2 * exp2i((CENTRED ? 9 : 24) - e);
            s *= p.qk2;
#pragma unroll
            for (int k = 0; k < 2; ++k) {   // rows 2c and 2c + 1
                sum[nt][k] = __shfl_sync(0xffffffffu, s, 8 * c + 4 * k);
                mul[nt][k] = __shfl_sync(0xffffffffu, back, 8 * c + 4 * k);
            }
        }
    }
};

// Scores of 16 tokens (rows 16 mt .. of the stage) in log2 units, less the
// column's `ref`: x[nt][0, 1] token r, columns 2c and 2c + 1; x[nt][2, 3]
// token r + 8.
template <int D, bool BF16, int NT, bool CENTRED>
__device__ __forceinline__ void scores(uint32_t stage, uint32_t par, int mt, const Queries<D, BF16, NT, CENTRED> &q,
                                       const float (&ref)[NT][2], float (&x)[NT][4])
{
    using L = Layout<D>;
    const int lane = threadIdx.x % 32, r = lane / 4, c = lane % 4;
    const uint32_t a0 = stage + (uint32_t)((16 * mt + r) * L::kRow + c * (L::kWords * 4));
    uint32_t wa[L::kWords], wb[L::kWords];
    if constexpr (D == 128) {
        const uint4 u = lds128(a0), v = lds128(a0 + 8 * L::kRow);
        wa[0] = u.x; wa[1] = u.y; wa[2] = u.z; wa[3] = u.w;
        wb[0] = v.x; wb[1] = v.y; wb[2] = v.z; wb[3] = v.w;
    } else {
        const uint2 u = lds64(a0), v = lds64(a0 + 8 * L::kRow);
        wa[0] = u.x; wa[1] = u.y;
        wb[0] = v.x; wb[1] = v.y;
    }
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
    for (int w = 0; w < L::kWords; ++w) {
        const uint32_t ya = wa[w] >> 8, yb = wb[w] >> 8;
        auto even = [](uint32_t v) { return CENTRED ? centred_even(v) : v & kEven; };
        auto odd = [](uint32_t v) { return CENTRED ? centred_odd(v) : v & kOdd; };
        const uint32_t lo[4] = {even(wa[w]), even(wb[w]), odd(wa[w]), odd(wb[w])};
        const uint32_t hi[4] = {even(ya), even(yb), odd(ya), odd(yb)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            mma(s[nt], lo, q.f[nt][2 * w][0], q.f[nt][2 * w][1]);
            mma(s[nt], hi, q.f[nt][2 * w + 1][0], q.f[nt][2 * w + 1][1]);
        }
    }
    const uint32_t pa = lds32(par + (uint32_t)(16 * mt + r) * 4), pb = lds32(par + (uint32_t)(16 * mt + r + 8) * 4);
    const float sa = to_float<BF16>(pa & 0xffffu), sb = to_float<BF16>(pb & 0xffffu);
    float za = to_float<BF16>(pa >> 16), zb = to_float<BF16>(pb >> 16);
    if (CENTRED) {
        za = fmaf(7.5f, sa, za);
        zb = fmaf(7.5f, sb, zb);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        x[nt][0] = fmaf(s[nt][0] * q.mul[nt][0], sa, fmaf(za, q.sum[nt][0], -ref[nt][0]));
        x[nt][1] = fmaf(s[nt][1] * q.mul[nt][1], sa, fmaf(za, q.sum[nt][1], -ref[nt][1]));
        x[nt][2] = fmaf(s[nt][2] * q.mul[nt][0], sb, fmaf(zb, q.sum[nt][0], -ref[nt][0]));
        x[nt][3] = fmaf(s[nt][3] * q.mul[nt][1], sb, fmaf(zb, q.sum[nt][1], -ref[nt][1]));
    }
}

// The tokens that the query of row n of a tile (row r0 + n of the key head)
// sees: [lo, hi), and those before `sink` that are before hi.
struct Bounds {
    int lo, hi, sink;
};

__device__ __forceinline__ Bounds bounds_of(const Params &p, int len, int row)
{
    Bounds v;
    const int i = row % p.Nq;
    const int pos = len - p.Nq + i;   // may be negative: sees nothing
    v.hi = pos + 1 < 0 ? 0 : pos + 1;
    v.lo = 0;
    v.sink = 0;
    if (p.left >= 0 && pos > p.left) {
        v.lo = pos - p.left;
        v.sink = p.sinks < v.hi ? p.sinks : v.hi;
    }
    return v;
}

__device__ __forceinline__ bool sees(const Bounds &v, int t)
{
    return (t >= v.lo && t < v.hi) || t < v.sink;
}

// One segment (units [ku, ke) of one tile) of the attention by one warp:
// running m, l, z = sum p vmin and O^T per query row.  O^T is formed from
// w = p vs as one fp16 operand: w is multiplied by the warp's power of two
// `fac`, which keeps the largest vs so far in [2^5, 2^6), so with p <= 2^8 it
// stays in fp16's range, and a token's 11 significand bits are whole down to
// 2^-20 of that.  Next to a bf16 result's rounding w's does not show (1.7e-3
// against float64 with and without it).  For an fp16 result, whose own
// rounding is as fine, w is two fp16 operands, the second what the first left
// out (3.7e-4 with one, 2.1e-4 with two, 2.1e-4 from the result's rounding
// alone): 8 more MMAs per 16 tokens at D = 128.  l is summed from the
// unrounded p.
template <int D, bool BF16, int NT>
struct Attend {
    using L = Layout<D>;
    float m[NT][2], l[NT][2], z[NT][2];
    float o[NT][L::kMTiles][4];
    float fac;

    __device__ void reset()
    {
        fac = exp2i(100);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[nt][e] = -INFINITY;
                l[nt][e] = z[nt][e] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < L::kMTiles; ++j)
                o[nt][j][0] = o[nt][j][1] = o[nt][j][2] = o[nt][j][3] = 0.f;
        }
    }

    // 32 tokens from t0 on, in `stage`; MASKED: some are hidden from some row.
    template <bool MASKED>
    __device__ __forceinline__ void step(uint32_t stage, const Queries<D, BF16, NT, false> &q, int t0,
                                         const Bounds (&vis)[NT][2])
    {
        const int lane = threadIdx.x % 32, r = lane / 4, c = lane % 4;
        const uint32_t par = stage + 2 * L::kCodes;
        float ref[NT][2];   // what the scores below are relative to
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                ref[nt][e] = m[nt][e] == -INFINITY ? 0.f : m[nt][e];
        float x[2][NT][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
            scores<D, BF16, NT, false>(stage, par, mt, q, ref, x[mt]);
        float vs[4], vm[4];   // scale and minimum of tokens r, r + 8, r + 16, r + 24
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t w = lds32(par + (uint32_t)(kSub + 8 * k + r) * 4);
            vs[k] = to_float<BF16>(w & 0xffffu);
            vm[k] = to_float<BF16>(w >> 16);
        }
        uint32_t hid = 0;   // (token, column) pairs that are hidden
        if (MASKED) {
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!sees(vis[nt][e & 1], t0 + 16 * mt + r + 8 * (e >> 1))) {
                            x[mt][nt][e] = -INFINITY;
                            hid |= 1u << ((mt * NT + nt) * 4 + e);
                        }
        }
        // Move the reference maxima where a score is kSlack above them (always
        // at the first visible token), and the factor of w where a scale has
        // outgrown it.
        bool up = false;
        float mx[NT][2], big = fmaxf(fmaxf(vs[0], vs[1]), fmaxf(vs[2], vs[3]));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mx[nt][e] = fmaxf(fmaxf(x[0][nt][e], x[0][nt][e + 2]), fmaxf(x[1][nt][e], x[1][nt][e + 2]));
                up |= mx[nt][e] > (m[nt][e] == -INFINITY ? -INFINITY : kSlack);
            }
        up |= big * fac >= 64.f;
        if (__any_sync(0xffffffffu, up)) {
            if (MASKED) {   // only rows that some query sees move the factor
                big = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    bool seen = false;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        seen |= ((hid >> (((k >> 1) * NT + nt) * 4 + 2 * (k & 1))) & 3u) != 3u;
                    big = fmaxf(big, seen ? vs[k] : 0.f);
                }
            }
            big = big < INFINITY ? big : 0.f;   // (and an infinite scale none but its own token's weight)
#pragma unroll
            for (int s = 4; s < 32; s *= 2)
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, s));
#pragma unroll
            for (int s = 1; s < 4; s *= 2)   // (masked: the columns of a token's lanes differ)
                big = MASKED ? fmaxf(big, __shfl_xor_sync(0xffffffffu, big, s)) : big;
            float df = 1.f;
            if (big * fac >= 64.f) {
                const int e = 5 + 127 - (int)(__float_as_uint(big) >> 23);   // big in [2^(5 - e), 2^(6 - e))
                const float now = exp2i(e > 100 ? 100 : (e < -125 ? -125 : e));
                df = now / fac;   // a power of two, or 0 from 2^100
                fac = now;
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int s = 4; s < 32; s *= 2)
                        mx[nt][e] = fmaxf(mx[nt][e], __shfl_xor_sync(0xffffffffu, mx[nt][e], s));
                    const bool first = m[nt][e] == -INFINITY;
                    // how far the reference moves (from ref = 0 at first: to the maximum itself)
                    const float by = mx[nt][e] == -INFINITY ? 0.f : (first ? mx[nt][e] : fmaxf(mx[nt][e], 0.f));
                    const float al = first ? 0.f : ex2(-by);
                    if (mx[nt][e] > -INFINITY)
                        m[nt][e] = ref[nt][e] + by;
                    l[nt][e] *= al;
                    z[nt][e] *= al;
#pragma unroll
                    for (int j = 0; j < L::kMTiles; ++j) {
                        o[nt][j][e] *= al * df;
                        o[nt][j][e + 2] *= al * df;
                    }
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        x[mt][nt][e] -= by;
                        x[mt][nt][e + 2] -= by;
                    }
                }
        }
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
            uint32_t wf[NT][2], wl[NT][2];   // w as B fragments; fp16 results: what they leave out
            const float wa = vs[2 * mt] * fac, wb = vs[2 * mt + 1] * fac;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float pr = ex2(x[mt][nt][e]);
                    l[nt][e & 1] += pr;
                    w[e] = pr * ((e >> 1) ? wb : wa);
                    if (MASKED) {   // a hidden token weighs nothing whatever its row holds
                        const bool h = (hid >> ((mt * NT + nt) * 4 + e)) & 1u;
                        w[e] = h ? 0.f : w[e];
                        z[nt][e & 1] = h ? z[nt][e & 1] : fmaf(pr, vm[2 * mt + (e >> 1)], z[nt][e & 1]);
                    } else {
                        z[nt][e & 1] = fmaf(pr, vm[2 * mt + (e >> 1)], z[nt][e & 1]);
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t u = pack_f16(w[2 * h], w[2 * h + 1]);
                    wf[nt][h] = transpose8(u);
                    if (!BF16)
                        wl[nt][h] = transpose8(pack_f16(w[2 * h] - to_float<false>(u & 0xffffu),
                                                        w[2 * h + 1] - to_float<false>(u >> 16)));
                }
            }
            // V^T as the A operand: for channel words of this lane, tokens
            // (2c, 2c + 1) and (2c + 8, 2c + 9).
            uint32_t vw[4][L::kVWords];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = 16 * mt + 8 * (k >> 1) + 2 * c + (k & 1);
                if constexpr (D == 128) {
                    const uint2 u = lds64(stage + L::kCodes + v_chunk<D>(t, r >> 1) + (r & 1) * 8);
                    vw[k][0] = u.x;
                    vw[k][1] = u.y;
                } else {
                    vw[k][0] = lds32(stage + L::kCodes + v_chunk<D>(t, r >> 2) + (r & 3) * 4);
                }
            }
#pragma unroll
            for (int w = 0; w < L::kVWords; ++w) {
                const uint32_t a0 = __byte_perm(vw[0][w], vw[1][w], 0x5410), a1 = __byte_perm(vw[0][w], vw[1][w], 0x7632);
                const uint32_t a2 = __byte_perm(vw[2][w], vw[3][w], 0x5410), a3 = __byte_perm(vw[2][w], vw[3][w], 0x7632);
                const uint32_t b0 = a0 >> 8, b1 = a1 >> 8, b2 = a2 >> 8, b3 = a3 >> 8;
                auto tile = [&](int j, const uint32_t (&a)[4]) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma(o[nt][j], a, wf[nt][0], wf[nt][1]);
                        if (!BF16)
                            mma(o[nt][j], a, wl[nt][0], wl[nt][1]);
                    }
                };
                tile(4 * w, {a0 & kEven, a1 & kEven, a2 & kEven, a3 & kEven});
                tile(4 * w + 1, {a0 & kOdd, a1 & kOdd, a2 & kOdd, a3 & kOdd});
                tile(4 * w + 2, {b0 & kEven, b1 & kEven, b2 & kEven, b3 & kEven});
                tile(4 * w + 3, {b0 & kOdd, b1 & kOdd, b2 & kOdd, b3 & kOdd});
            }
        }
    }

    // sum_t p_t vs_t code_t of an accumulator of tile j.
    __device__ float value(int j, float acc) const
    {
        return acc * ((j & 1) ? kCodeUnit / 16.f : kCodeUnit) * (1.f / fac);
    }
};

// Channel of row half h (0: r, 1: r + 8) of O^T tile j of lane row r.
template <int D>
__device__ __forceinline__ int out_channel(int r, int j, int h)
{
    return r * (D / 8) + 8 * (j / 4) + 4 * h + j % 4;
}

template <int D, int NT>
struct AttendSmem {
    static constexpr int kPipe = kWarps * kStages * Layout<D>::kStage;
    static constexpr int kORow = D + 4;                                  // fp32 row of a warp's O, padded
    static constexpr int kJoin = kWarps * 8 * NT * (kORow * 4 + 8);      // O, then (m, l), of every warp
    static constexpr int kArea = kPipe > kJoin ? kPipe : kJoin;
    static constexpr int kScratch = (kWarps + 2) * 8;
    static constexpr int kBytes = kArea + kScratch;
};

// O = acc / l and LSE of one row's channels [ch, ch + 4).
template <int D, bool BF16>
__device__ __forceinline__ void store_out(const Params &p, long long row, int ch, const float (&v)[4], float M, float Lsum)
{
    const float inv = Lsum != 0.f ? 1.f / Lsum : 0.f;   // a row that sees nothing: O = 0, LSE = -inf (NaN stays NaN)
    uint2 w;
    w.x = from_float<BF16>(v[0] * inv) | (from_float<BF16>(v[1] * inv) << 16);
    w.y = from_float<BF16>(v[2] * inv) | (from_float<BF16>(v[3] * inv) << 16);
    *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(p.o) + row * D + ch) = w;
    if (ch == 0)
        p.lse[row] = Lsum != 0.f ? (M + log2f(Lsum)) * kLn2f : -INFINITY;
}

// Persistent CTAs; CTA c of G runs units [U c / G, U (c + 1) / G) of the
// ordered tiles (sequence, key head, row block), so every CTA reads the same
// number of tokens whatever the lengths are.  A tile's first and last share
// may be partial (slots 2c, 2c + 1); merge_kernel joins those.  Within a CTA
// the eight warps take 32-token steps in turn, each through its own ring of
// cp.async stages, so no barrier stands between loads and products; they join
// their running sums through shared memory at the end of a tile.  Where `whole`
// is set the CTAs share out whole tiles instead.
template <int D, bool BF16, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) attend_kernel(const Params p)
{
    using L = Layout<D>;
    using S = AttendSmem<D, NT>;
    extern __shared__ __align__(128) uint8_t smem[];
    launch_dependents();
    long long *scratch = reinterpret_cast<long long *>(smem + S::kArea);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, r = lane / 4, c = lane % 4;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + (uint32_t)(warp * kStages * L::kStage);

    const int HR = p.Hkv * p.RB;
    long long u0, u1;   // units, or tiles where none is cut
    int b, hr, ku = 0;
    Span sp;
    if (p.whole) {
        const long long tiles = (long long)p.B * HR;
        u0 = tiles * blockIdx.x / gridDim.x;
        u1 = tiles * (blockIdx.x + 1) / gridDim.x;
        if (u0 == u1)
            return;
        b = (int)(u0 / HR);
        hr = (int)(u0 - (long long)b * HR);
        sp = span_of(p, b);
    } else {
        const Where w = locate(p, blockIdx.x, gridDim.x, scratch);
        if ((long long)blockIdx.x >= w.parts)
            return;
        u0 = w.first;
        u1 = w.total * (blockIdx.x + 1) / w.parts;
        b = w.b;
        sp = span_of(p, b);
        hr = (int)((u0 - w.before) / sp.n);
        ku = (int)((u0 - w.before) - (long long)hr * sp.n);
    }

    for (long long u = u0; u < u1;) {
        const int ke = p.whole || (long long)sp.n - ku < u1 - u ? sp.n : (int)(ku + (u1 - u));
        const bool whole = ku == 0 && ke == sp.n;
        const int h = hr / p.RB, r0 = (hr - h * p.RB) * (8 * NT);
        const int nrows = p.rows - r0 < 8 * NT ? p.rows - r0 : 8 * NT;
        const long long bh = (long long)b * p.Hkv + h;
        const long long row0 = bh * p.rows + r0;   // of the [B H Nq] query rows

        const Rows<D> rows(p, bh);
        const int nsub = (ke - ku) * (kUnit / kSub);
        auto token = [&](int s) { return sp.token(ku + s / (kUnit / kSub)) + (s % (kUnit / kSub)) * kSub; };
        // Two stages ahead; the query rows load behind them.
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) {
            const int s = warp + i * kWarps;
            load_stage<D, true>(rows, ring + i * L::kStage, s < nsub ? token(s) : 0, sp.len, s < nsub);
        }
        Queries<D, BF16, NT, false> q;
        q.load(p, row0, nrows);
        Bounds vis[NT][2];
        int edge_lo = 0, edge_hi = 0x7fffffff;   // tokens in [edge_lo, edge_hi) are seen by every row
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int n = 8 * nt + 2 * c + e;
                vis[nt][e] = bounds_of(p, sp.len, r0 + (n < nrows ? n : nrows - 1));
                edge_lo = max(edge_lo, vis[nt][e].lo);
                edge_hi = min(edge_hi, vis[nt][e].hi);
            }
#pragma unroll
        for (int s = 1; s < 4; s *= 2) {
            edge_lo = max(edge_lo, __shfl_xor_sync(0xffffffffu, edge_lo, s));
            edge_hi = min(edge_hi, __shfl_xor_sync(0xffffffffu, edge_hi, s));
        }
        Attend<D, BF16, NT> a;
        a.reset();
        int st = 0;
        for (int s = warp; s < nsub; s += kWarps) {
            cp_wait<kStages - 2>();
            __syncwarp();   // the step's tokens are here, and every lane is done with the stage refilled below
            const int next = s + (kStages - 1) * kWarps;
            const int fill = st + kStages - 1 >= kStages ? st - 1 : st + kStages - 1;
            load_stage<D, true>(rows, ring + fill * L::kStage, next < nsub ? token(next) : 0, sp.len, next < nsub);
            const int t0 = token(s);
            if (t0 < edge_lo || t0 + kSub > edge_hi)
                a.template step<true>(ring + st * L::kStage, q, t0, vis);
            else
                a.template step<false>(ring + st * L::kStage, q, t0, vis);
            st = st + 1 == kStages ? 0 : st + 1;
        }
        cp_wait<0>();
        __syncthreads();   // every warp is done with its ring: the area is reused below

        // Per warp: l and z summed over the lanes' tokens, z added to every channel.
        float *jo = reinterpret_cast<float *>(smem) + (size_t)warp * 8 * NT * S::kORow;
        float2 *jml = reinterpret_cast<float2 *>(smem + (size_t)kWarps * 8 * NT * S::kORow * 4) + warp * 8 * NT;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = a.l[nt][e], z = a.z[nt][e];
#pragma unroll
                for (int s = 4; s < 32; s *= 2) {
                    l += __shfl_xor_sync(0xffffffffu, l, s);
                    z += __shfl_xor_sync(0xffffffffu, z, s);
                }
                const int n = 8 * nt + 2 * c + e;
                if (r == 0)
                    jml[n] = make_float2(a.m[nt][e], l);
#pragma unroll
                for (int j = 0; j < L::kMTiles; ++j) {
                    jo[n * S::kORow + out_channel<D>(r, j, 0)] = a.value(j, a.o[nt][j][e]) + z;
                    jo[n * S::kORow + out_channel<D>(r, j, 1)] = a.value(j, a.o[nt][j][e + 2]) + z;
                }
            }
        __syncthreads();
        {
            const float *all_o = reinterpret_cast<const float *>(smem);
            const float2 *all_ml = reinterpret_cast<const float2 *>(smem + (size_t)kWarps * 8 * NT * S::kORow * 4);
            for (int i = threadIdx.x; i < 8 * NT * (D / 4); i += kThreads) {
                const int n = i / (D / 4), ch = (i % (D / 4)) * 4;
                if (n >= nrows)
                    continue;
                float M = -INFINITY;
#pragma unroll
                for (int k = 0; k < kWarps; ++k)
                    M = fmaxf(M, all_ml[k * 8 * NT + n].x);
                float Lsum = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < kWarps; ++k) {
                    const float2 ml = all_ml[k * 8 * NT + n];
                    const float f = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : ex2(ml.x - M);
                    const float4 x = *reinterpret_cast<const float4 *>(all_o + (size_t)(k * 8 * NT + n) * S::kORow + ch);
                    Lsum += ml.y * f;
                    v[0] += x.x * f;
                    v[1] += x.y * f;
                    v[2] += x.z * f;
                    v[3] += x.w * f;
                }
                if (whole) {
                    store_out<D, BF16>(p, row0 + n, ch, v, M, Lsum);
                } else {
                    const long long slot = 2ll * blockIdx.x + (u == u0 ? 0 : 1);
                    *reinterpret_cast<float4 *>(p.part_o + (slot * 8 * NT + n) * D + ch) = make_float4(v[0], v[1], v[2], v[3]);
                    if (ch == 0)
                        p.part_ml[slot * 8 * NT + n] = make_float2(M, Lsum);
                }
            }
        }
        __syncthreads();   // read before the next tile's loads overwrite it
        u += p.whole ? 1 : ke - ku;
        ku = 0;
        if (++hr == HR && u < u1) {
            hr = 0;
            sp = span_of(p, ++b);
        }
    }
}

// Joins the parts of the tiles that a share boundary cuts: block k looks at
// the boundary between CTAs k and k + 1 and, if it is the first one inside its
// tile, adds that tile's parts in order (so the result does not depend on
// which CTA finished first).
template <int D, bool BF16, int NT>
__global__ void __launch_bounds__(kThreads) merge_kernel(const Params p, int grid)
{
    __shared__ long long scratch[kWarps + 2];
    // (lens are inputs: the search may run before the attention has ended)
    const int k = blockIdx.x;
    const Where w = locate_quick(p, k + 1, grid, scratch);
    grid_wait();   // by every block, so that this grid ends after the attention has
    const long long G = w.parts, U = w.total;
    if (k + 1 >= G)
        return;
    const long long edge = w.first;   // first unit of CTA k + 1
    const Span sp = span_of(p, w.b);
    const int hr = tile_of(edge - w.before, sp.n);
    const long long t0 = w.before + (long long)hr * sp.n, t1 = t0 + sp.n;   // the tile's units
    const long long start = share_of(w, k);   // of CTA k's units
    if (t0 == edge || start > t0)   // not inside a tile, or not its first boundary
        return;
    const long long last = (t1 * G - 1) / U;   // CTA holding unit t1 - 1: the largest x with U x / G < t1
    const int h = hr / p.RB, r0 = (hr - h * p.RB) * (8 * NT);
    const int nrows = p.rows - r0 < 8 * NT ? p.rows - r0 : 8 * NT;
    const long long row0 = ((long long)w.b * p.Hkv + h) * p.rows + r0;
    const long long slot0 = 2 * k + (start == t0 ? 0 : 1);   // CTA k's part: its only one, or its last
    for (int i = threadIdx.x; i < nrows * (D / 4); i += kThreads) {
        const int n = i / (D / 4), ch = (i % (D / 4)) * 4;
        float M = -INFINITY;
        for (long long x = k; x <= last; ++x)
            M = fmaxf(M, p.part_ml[(x == k ? slot0 : 2 * x) * 8 * NT + n].x);
        float Lsum = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (long long x = k; x <= last; ++x) {
            const long long at = (x == k ? slot0 : 2 * x) * 8 * NT + n;
            const float2 ml = p.part_ml[at];
            const float f = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : ex2(ml.x - M);
            const float4 y = *reinterpret_cast<const float4 *>(p.part_o + at * D + ch);
            Lsum += ml.y * f;
            v[0] += y.x * f;
            v[1] += y.y * f;
            v[2] += y.z * f;
            v[3] += y.w * f;
        }
        store_out<D, BF16>(p, row0 + n, ch, v, M, Lsum);
    }
}

// ------------------------------------------------------------------ weights

// The entries of acc that no unit holds, by the CTA that runs the tile's first
// unit (between the sinks and the window) or its last (past the sequence).
__device__ __forceinline__ void zero_rest(const Params &p, float *acc, const Span &sp, int ku, int ke)
{
    if (ku == 0)
        for (int t = sp.su * kUnit + threadIdx.x; t < sp.ks * kUnit && t < sp.len; t += kThreads)
            acc[t] = 0.f;
    if (ke == sp.n)
        for (int t = sp.len + threadIdx.x; t < p.C; t += kThreads)
            acc[t] = 0.f;
}

// acc[b, h, t] (+)= sum over the key head's query rows of exp(x_t - LSE): the
// scores again, K alone, with the LSE that the attention returned.  A token's
// sum is formed by one warp, in a fixed order, and every entry of acc has one
// writer, so nothing is added by atomics.  This kernel takes up to 8 NT query
// rows, held as fragments in registers (decoding); more go to fa_cache_rows.cu.
template <int D, bool BF16, int NT>
__global__ void __launch_bounds__(kThreads, 2) weights_kernel(const Params p)
{
    using L = Layout<D>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long scratch[kWarps + 2];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, r = lane / 4, c = lane % 4;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + (uint32_t)(warp * kStages * L::kKeyStage);
    const Where w = locate_quick(p, blockIdx.x, gridDim.x, scratch);
    if ((long long)blockIdx.x >= w.parts)
        return;
    const long long u0 = w.first, u1 = share_of(w, blockIdx.x + 1);
    int b = w.b;
    Span sp = span_of(p, b);
    int h = tile_of(u0 - w.before, sp.n);
    int ku = (int)((u0 - w.before) - (long long)h * sp.n);
    for (long long u = u0; u < u1;) {
        const int ke = (int)((long long)sp.n - ku < u1 - u ? sp.n : ku + (u1 - u));
        const long long bh = (long long)b * p.Hkv + h;
        float *acc = p.acc + bh * p.C;
        const Rows<D> rows(p, bh);
        const int nsub = (ke - ku) * (kUnit / kSub);
        auto token = [&](int s) { return sp.token(ku + s / (kUnit / kSub)) + (s % (kUnit / kSub)) * kSub; };
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) {
            const int s = warp + i * kWarps;
            load_stage<D, false>(rows, ring + i * L::kKeyStage, s < nsub ? token(s) : 0, sp.len, s < nsub);
        }
        Queries<D, BF16, NT, true> q;
        q.load(p, bh * p.rows, p.rows);
        Bounds vis[NT][2];
        // LSE in log2 units, what the scores are taken relative to, and 2 to the
        // power of what its rounding to fp32 left out (1 + 1e-6 at most, but the
        // same for a whole row); +inf for rows that are not there or see nothing
        float ref[NT][2], rest[NT][2];
        int edge_lo = 0, edge_hi = 0x7fffffff;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int n = 8 * nt + 2 * c + e;
                const float lse = n < p.rows ? p.lse[bh * p.rows + n] : -INFINITY;
                ref[nt][e] = lse == -INFINITY ? INFINITY : lse * kLog2e;
                rest[nt][e] = lse == -INFINITY ? 1.f : exp2f(-fmaf(lse, kLog2e, -ref[nt][e]) - lse * kLog2eRest);
                vis[nt][e] = bounds_of(p, sp.len, n < p.rows ? n : p.rows - 1);
                edge_lo = max(edge_lo, vis[nt][e].lo);
                edge_hi = min(edge_hi, vis[nt][e].hi);
            }
#pragma unroll
        for (int s = 1; s < 4; s *= 2) {
            edge_lo = max(edge_lo, __shfl_xor_sync(0xffffffffu, edge_lo, s));
            edge_hi = min(edge_hi, __shfl_xor_sync(0xffffffffu, edge_hi, s));
        }
        int st = 0;
        for (int s = warp; s < nsub; s += kWarps) {
            cp_wait<kStages - 2>();
            __syncwarp();
            const int next = s + (kStages - 1) * kWarps;
            const int fill = st + kStages - 1 >= kStages ? st - 1 : st + kStages - 1;
            load_stage<D, false>(rows, ring + fill * L::kKeyStage, next < nsub ? token(next) : 0, sp.len, next < nsub);
            const int t0 = token(s);
            const bool masked = t0 < edge_lo || t0 + kSub > edge_hi;
            const uint32_t stage = ring + st * L::kKeyStage;
            float sum[4];   // tokens r, r + 8, r + 16, r + 24
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                float x[NT][4];
                scores<D, BF16, NT, true>(stage, stage + L::kCodes, mt, q, ref, x);
                if (masked) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!sees(vis[nt][e & 1], t0 + 16 * mt + r + 8 * (e >> 1)))
                                x[nt][e] = -INFINITY;
                }
                // (rows that are not there or see nothing: -inf, so 0)
                sum[2 * mt] = sum[2 * mt + 1] = 0.f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sum[2 * mt + (e >> 1)] = fmaf(ex2(x[nt][e]), rest[nt][e & 1], sum[2 * mt + (e >> 1)]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 1);
                sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 2);
            }
            // lane (r, c) writes token r + 8 c
            const float mine = c == 0 ? sum[0] : (c == 1 ? sum[1] : (c == 2 ? sum[2] : sum[3]));
            const int t = t0 + r + 8 * c;
            if (t < sp.len)
                acc[t] = p.accumulate ? acc[t] + mine : mine;
            st = st + 1 == kStages ? 0 : st + 1;
        }
        cp_wait<0>();
        __syncwarp();
        if (!p.accumulate)
            zero_rest(p, acc, sp, ku, ke);
        u += ke - ku;
        ku = 0;
        if (++h == p.Hkv && u < u1) {
            h = 0;
            sp = span_of(p, ++b);
        }
    }
}

}  // namespace cache
}  // namespace fa
