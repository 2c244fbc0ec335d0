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
// (exact, the input) and against w_j = p_j vs_j.
//
// What bounds it: a decoded token reads every visible row once, D/2 + 4 bytes
// for each of K and V, and does 4 G Nq D operations on it -- HBM, at the few
// query rows per key head of decoding, if unpacking keeps up: 64 codes per
// lane and 16 tokens for each of K and V, about one integer operation each.
// Hence mma.sync and not tcgen05: the codes go from shared memory through
// registers (unpacking) straight into A fragments (16 tokens or channels x 16)
// with the 8 query rows as the N dimension, where tcgen05 would want the
// unpacked operand written back to shared memory or TMEM first, and its M =
// 128 rows are 16 times what a decode step has.
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

// D[16 x 8] += A[16 x 16] B[16 x 8], fp32 accumulation.
template <bool BF16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
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

// Codes I and I + 4 of a word of eight as the 16-bit pair (16 + code I, 16 +
// code I + 4): the code goes to the top of the significand of 16.0, so one
// shift and one three-input logic operation unpack two codes.  The 16 is
// taken out of the finished sums (16 rather than a larger power keeps the
// sums, and with them fp32's rounding, small).
template <bool BF16, int I>
__device__ __forceinline__ uint32_t unpack2(uint32_t w)
{
    constexpr int up = (BF16 ? 3 : 6) - 4 * I;   // from bit 4 I to the significand's top four bits
    const uint32_t s = up >= 0 ? w << (up >= 0 ? up : 0) : w >> (up >= 0 ? 0 : -up);
    return (s & (BF16 ? 0x00780078u : 0x03C003C0u)) | (BF16 ? 0x41804180u : 0x4C004C00u);
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

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// ------------------------------------------------------------------ append, read

// What one row's codes are computed from: x (scaled by `k`, a power of two
// that keeps the differences and the scale inside fp32's normal range; 1 but
// for extreme rows), the scale and minimum likewise.
struct RowScale {
    float mn, sc, inv, k;
    uint32_t params;   // as held: scale, minimum
    bool flat;         // scale 0, or a row that is not finite: codes 0
};

template <bool BF16>
__device__ __forceinline__ RowScale row_scale(float mn, float mx, bool finite)
{
    RowScale r;
    r.k = 1.f;
    if (!finite) {   // an infinity or NaN in the row: every value it stands for is NaN
        r.params = BF16 ? 0x7FC07FC0u : 0x7E007E00u;
        r.flat = true;
        r.mn = r.sc = r.inv = 0.f;
        return r;
    }
    float range = mx - mn;
    if (range > 3.0e38f)   // (bf16) the range overflows: in quarters
        r.k = 0.25f;
    else if (range > 0.f && range < 8.0e-25f)
        r.k = 1.2089258196146292e24f;   // 2^80: the scale and its reciprocal stay normal
    if (r.k != 1.f)
        range = mx * r.k - mn * r.k;
    float sc = __fdiv_rn(range, 15.f);
    if (r.k == 1.f) {
        r.params = from_float<BF16>(sc);
    } else {
        r.params = from_float<BF16>(__fdiv_rn(sc, r.k));   // (exact but for a scale that ends subnormal)
    }
    const float held = to_float<BF16>(r.params);
    r.params |= from_float<BF16>(mn) << 16;
    r.flat = held == 0.f;
    r.sc = held * r.k;
    r.inv = r.flat ? 0.f : __fdiv_rn(1.f, r.sc);
    r.mn = mn * r.k;
    return r;
}

// round_half_even((x - mn) / sc) clamped to 0..15.  The quotient by the
// reciprocal is off by a few units in its last place, which matters only next
// to a border between two codes: there the residual a - (q -+ 1/2) sc decides,
// with the rounding error of a = x - mn added back.
__device__ __forceinline__ uint32_t code_of(float x, const RowScale &r)
{
    const float a = x - r.mn;
    const float f = a * r.inv;
    float q = rintf(f);
    if (fabsf(f - q) > 0.4999f) {
        const float bb = a - x;
        const float e = (x - (a - bb)) + (-r.mn - bb);
        const float t = fmaf(-q, r.sc, a);
        if (f > q) {
            const float over = (t - 0.5f * r.sc) + e;
            if (over > 0.f || (over == 0.f && ((int)q & 1)))
                q += 1.f;
        } else {
            const float under = (t + 0.5f * r.sc) + e;
            if (under < 0.f || (under == 0.f && ((int)q & 1)))
                q -= 1.f;
        }
    }
    return (uint32_t)fminf(fmaxf(q, 0.f), 15.f);
}

// Position of new token i of sequence b in the cache, or -1: not counted in,
// or outside [0, C).
__device__ __forceinline__ int slot_of(const int *start, const int *count, int b, int i, int N, int C)
{
    const int n = count ? count[b] : N;
    const long long at = (long long)start[b] + i;
    return (i < n && at >= 0 && at < C) ? (int)at : -1;
}

template <int D, bool BF16>
__device__ __forceinline__ void append_row(const uint4 &x4, int part, uint32_t group, uint8_t *codes, uint32_t *params)
{
    const uint32_t xw[4] = {x4.x, x4.y, x4.z, x4.w};
    float x[8];
    float mn = INFINITY, mx = -INFINITY, zero = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = to_float<BF16>((i & 1) ? xw[i / 2] >> 16 : xw[i / 2] & 0xffffu);
        mn = fminf(mn, x[i]);
        mx = fmaxf(mx, x[i]);
        zero = fmaf(x[i], 0.f, zero);   // NaN once an element is not finite
    }
#pragma unroll
    for (int m = D / 16; m > 0; m /= 2) {
        mn = fminf(mn, __shfl_xor_sync(group, mn, m));
        mx = fmaxf(mx, __shfl_xor_sync(group, mx, m));
        zero += __shfl_xor_sync(group, zero, m);
    }
    const RowScale r = row_scale<BF16>(mn, mx, zero == 0.f);
    uint32_t w = 0;
    if (!r.flat) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w |= code_of(x[i] * r.k, r) << (4 * i);
    }
    *reinterpret_cast<uint32_t *>(codes + part * 4) = w;
    if (part == 0)
        *params = r.params;
}

// One group of D / 8 lanes per new token and head, K and V both (two loads in
// flight per lane), 8 channels a lane.  Bound by HBM: 2 x 2 D bytes read and
// 2 x (D/2 + 4) written per token and head.
template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads)
    append_kernel(const uint16_t *kn, const uint16_t *vn, uint8_t *kc, uint32_t *kp, uint8_t *vc, uint32_t *vp,
                  const int *start, const int *count, int Hkv, int N, int C, long long rows)
{
    constexpr int kTpr = D / 8;
    const long long g = (long long)blockIdx.x * kThreads + threadIdx.x;
    const long long row = g / kTpr;
    if (row >= rows)   // whole groups leave together
        return;
    const int part = (int)(g % kTpr);
    const long long bh = row / N;
    const int i = (int)(row - bh * N);
    const int at = slot_of(start, count, (int)(bh / Hkv), i, N, C);
    if (at < 0)
        return;
    const uint4 k4 = __ldg(reinterpret_cast<const uint4 *>(kn + row * D) + part);
    const uint4 v4 = __ldg(reinterpret_cast<const uint4 *>(vn + row * D) + part);
    const int lane = threadIdx.x % 32;
    const uint32_t group = ((1u << kTpr) - 1u) << (lane & ~(kTpr - 1));
    const long long dst = bh * C + at;
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
        const float lo = fmaf((float)((w >> (8 * i)) & 15u), sc, mn), hi = fmaf((float)((w >> (8 * i + 4)) & 15u), sc, mn);
        o[i] = from_float<BF16>(lo) | (from_float<BF16>(hi) << 16);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// The values that rows start[b] .. start[b] + N - 1 stand for, rounded once
// to the cache's type; rows not counted in or outside the cache are zeros.
template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads)
    read_kernel(const uint8_t *kc, const uint32_t *kp, const uint8_t *vc, const uint32_t *vp, uint16_t *ko, uint16_t *vo,
                const int *start, const int *count, int Hkv, int N, int C, long long rows)
{
    constexpr int kTpr = D / 8;
    const long long g = (long long)blockIdx.x * kThreads + threadIdx.x;
    const long long row = g / kTpr;
    if (row >= rows)
        return;
    const int part = (int)(g % kTpr);
    const long long bh = row / N;
    const int i = (int)(row - bh * N);
    const int at = slot_of(start, count, (int)(bh / Hkv), i, N, C);
    uint4 k4 = make_uint4(0u, 0u, 0u, 0u), v4 = k4;
    if (at >= 0) {
        const long long src = bh * C + at;
        const uint32_t kw = *reinterpret_cast<const uint32_t *>(kc + src * (D / 2) + part * 4);
        const uint32_t vw = *reinterpret_cast<const uint32_t *>(vc + src * (D / 2) + part * 4);
        k4 = values_of<BF16>(kw, kp[src]);
        v4 = values_of<BF16>(vw, vp[src]);
    }
    reinterpret_cast<uint4 *>(ko + row * D)[part] = k4;
    reinterpret_cast<uint4 *>(vo + row * D)[part] = v4;
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

// Called by every thread of the block (it reads all of lens); `scratch` holds
// kWarps + 2 values.  Threads take consecutive sequences; an exclusive scan
// over the threads' sums, then the owning thread walks its own.
__device__ inline Where locate(const Params &p, int k, int grid, long long *scratch)
{
    const int t = threadIdx.x, lane = t % 32, warp = t / 32;
    const int per = (p.B + kThreads - 1) / kThreads;
    const long long HR = (long long)p.Hkv * p.RB;
    long long sum = 0;
    for (int i = t * per; i < (t + 1) * per && i < p.B; ++i)
        sum += span_of(p, i).n * HR;
    long long inc = sum;
#pragma unroll
    for (int m = 1; m < 32; m *= 2) {
        const long long v = __shfl_up_sync(0xffffffffu, inc, m);
        if (lane >= m)
            inc += v;
    }
    if (lane == 31)
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

// Issue the loads of tokens t0 .. t0 + 31 of key head `bh` into a stage (V
// left out for the weights); tokens from `len` on are zeros.  Always commits
// a group.
template <int D, bool VALUES>
__device__ __forceinline__ void load_stage(const Params &p, uint32_t stage, long long bh, int t0, int len, bool any)
{
    using L = Layout<D>;
    const int lane = threadIdx.x % 32;
    if (any) {
        constexpr int kPer = L::kRow / 16;   // 16-byte chunks per row
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int idx = lane + 32 * i, t = idx / kPer, j = idx % kPer;
            const bool real = t0 + t < len;
            const long long row = bh * p.C + (real ? t0 + t : 0);
            cp16(stage + idx * 16, p.kc + row * L::kRow + j * 16, real);
            if (VALUES)
                cp16(stage + L::kCodes + v_chunk<D>(t, j), p.vc + row * L::kRow + j * 16, real);
        }
        const bool real = t0 + lane < len;
        const long long row = bh * p.C + (real ? t0 + lane : 0);
        const uint32_t par = stage + (VALUES ? 2 : 1) * L::kCodes;
        cp4(par + lane * 4, p.kp + row, real);
        if (VALUES)
            cp4(par + (kSub + lane) * 4, p.vp + row, real);
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
// gives two fragments, (0, 4 | 1, 5) and (2, 6 | 3, 7).  Also -16 sum_d q_d
// and sum_d q_d per row, for the two rows (columns of S^T) of this lane.
template <int D, bool BF16, int NT>
struct Queries {
    using L = Layout<D>;
    uint32_t f[NT][L::kWords * 2][2];
    float sum[NT][2];

    __device__ void load(const Params &p, long long row0, int nrows)
    {
        const int lane = threadIdx.x % 32, r = lane / 4, c = lane % 4;
        const uint32_t *q = reinterpret_cast<const uint32_t *>(p.q);   // channel pairs
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int n = 8 * nt + r;
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < L::kWords; ++w) {
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (n < nrows)
                    x = __ldg(reinterpret_cast<const uint4 *>(q + (row0 + n) * (D / 2) + (c * L::kWords + w) * 4));
                const uint32_t xw[4] = {x.x, x.y, x.z, x.w};   // channels (0,1) (2,3) (4,5) (6,7)
                f[nt][2 * w][0] = __byte_perm(xw[0], xw[2], 0x5410);       // 0, 4
                f[nt][2 * w][1] = __byte_perm(xw[0], xw[2], 0x7632);       // 1, 5
                f[nt][2 * w + 1][0] = __byte_perm(xw[1], xw[3], 0x5410);   // 2, 6
                f[nt][2 * w + 1][1] = __byte_perm(xw[1], xw[3], 0x7632);   // 3, 7
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s += to_float<BF16>(xw[i] & 0xffffu) + to_float<BF16>(xw[i] >> 16);
            }
            s += __shfl_xor_sync(0xffffffffu, s, 1);
            s += __shfl_xor_sync(0xffffffffu, s, 2);
            sum[nt][0] = __shfl_sync(0xffffffffu, s, 8 * c);       // row 2c
            sum[nt][1] = __shfl_sync(0xffffffffu, s, 8 * c + 4);   // row 2c + 1
        }
    }
};

// Scores of 16 tokens (rows 16 mt .. of the stage) in log2 units: x[nt][0, 1]
// token r, columns 2c and 2c + 1; x[nt][2, 3] token r + 8.
template <int D, bool BF16, int NT>
__device__ __forceinline__ void scores(const Params &p, uint32_t stage, uint32_t par, int mt,
                                       const Queries<D, BF16, NT> &q, float (&x)[NT][4])
{
    using L = Layout<D>;
    const int lane = threadIdx.x % 32, r = lane / 4, c = lane % 4;
    const uint32_t a0 = stage + (uint32_t)((16 * mt + r) * L::kRow + c * (L::kWords * 4));
    uint32_t wa[L::kWords], wb[L::kWords];
    if constexpr (D == 128) {
        const uint4 u = lds128(a0), v = lds128(a0 + 8 * L::kRow);
        wa[0] = u.x; wa[1] = u.y; wa[L::kWords - 2] = u.z; wa[L::kWords - 1] = u.w;
        wb[0] = v.x; wb[1] = v.y; wb[L::kWords - 2] = v.z; wb[L::kWords - 1] = v.w;
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
        const uint32_t lo[4] = {unpack2<BF16, 0>(wa[w]), unpack2<BF16, 0>(wb[w]), unpack2<BF16, 1>(wa[w]),
                                unpack2<BF16, 1>(wb[w])};
        const uint32_t hi[4] = {unpack2<BF16, 2>(wa[w]), unpack2<BF16, 2>(wb[w]), unpack2<BF16, 3>(wa[w]),
                                unpack2<BF16, 3>(wb[w])};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            mma<BF16>(s[nt], lo, q.f[nt][2 * w][0], q.f[nt][2 * w][1]);
            mma<BF16>(s[nt], hi, q.f[nt][2 * w + 1][0], q.f[nt][2 * w + 1][1]);
        }
    }
    const uint32_t pa = lds32(par + (uint32_t)(16 * mt + r) * 4), pb = lds32(par + (uint32_t)(16 * mt + r + 8) * 4);
    const float sa = to_float<BF16>(pa & 0xffffu) * p.qk2, sb = to_float<BF16>(pb & 0xffffu) * p.qk2;
    const float za = fmaf(-16.f, sa, to_float<BF16>(pa >> 16) * p.qk2), zb = fmaf(-16.f, sb, to_float<BF16>(pb >> 16) * p.qk2);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        x[nt][0] = fmaf(sa, s[nt][0], za * q.sum[nt][0]);
        x[nt][1] = fmaf(sa, s[nt][1], za * q.sum[nt][1]);
        x[nt][2] = fmaf(sb, s[nt][2], zb * q.sum[nt][0]);
        x[nt][3] = fmaf(sb, s[nt][3], zb * q.sum[nt][1]);
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
// running m, l, z = sum p (vmin - 16 vs) and O^T per query row.
template <int D, bool BF16, int NT>
struct Attend {
    using L = Layout<D>;
    float m[NT][2], l[NT][2], z[NT][2];
    float o[NT][L::kMTiles][4];

    __device__ void reset()
    {
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

    // 32 tokens from t0 on, in `stage`.
    __device__ void step(const Params &p, uint32_t stage, const Queries<D, BF16, NT> &q, int t0, bool masked,
                         const Bounds (&vis)[NT][2])
    {
        const int lane = threadIdx.x % 32, r = lane / 4, c = lane % 4;
        const uint32_t par = stage + 2 * L::kCodes;
        float x[2][NT][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
            scores<D, BF16, NT>(p, stage, par, mt, q, x[mt]);
        if (masked) {
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!sees(vis[nt][e & 1], t0 + 16 * mt + r + 8 * (e >> 1)))
                            x[mt][nt][e] = -INFINITY;
        }
        // Move the reference maxima where a score is kSlack above them (always
        // at the first visible token).
        bool up = false;
        float mx[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mx[nt][e] = fmaxf(fmaxf(x[0][nt][e], x[0][nt][e + 2]), fmaxf(x[1][nt][e], x[1][nt][e + 2]));
                up |= mx[nt][e] > m[nt][e] + kSlack;
            }
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int s = 4; s < 32; s *= 2)
                        mx[nt][e] = fmaxf(mx[nt][e], __shfl_xor_sync(0xffffffffu, mx[nt][e], s));
                    const float mn = fmaxf(m[nt][e], mx[nt][e]);
                    const float al = mn == m[nt][e] ? 1.f : ex2(m[nt][e] - mn);   // 0 from m = -inf
                    m[nt][e] = mn;
                    l[nt][e] *= al;
                    z[nt][e] *= al;
#pragma unroll
                    for (int j = 0; j < L::kMTiles; ++j) {
                        o[nt][j][e] *= al;
                        o[nt][j][e + 2] *= al;
                    }
                }
        }
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
            // Weights of the V codes, w = p vs, as bf16 pairs hi + lo (16 bits
            // of significand together: one bf16 alone would put 2^-9 of error
            // on every weight, more than a half-precision output's own
            // rounding): 4 more MMAs per 16 tokens and 64 channels.
            const uint32_t pa = lds32(par + (uint32_t)(kSub + 16 * mt + r) * 4),
                           pb = lds32(par + (uint32_t)(kSub + 16 * mt + r + 8) * 4);
            const float va[2] = {to_float<BF16>(pa & 0xffffu), to_float<BF16>(pb & 0xffffu)};
            const float vb[2] = {fmaf(-16.f, va[0], to_float<BF16>(pa >> 16)), fmaf(-16.f, va[1], to_float<BF16>(pb >> 16))};
            uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float mu = m[nt][e & 1];
                    const float pr = ex2(x[mt][nt][e] - (mu == -INFINITY ? 0.f : mu));
                    l[nt][e & 1] += pr;
                    // (a hidden token weighs nothing whatever its row holds)
                    w[e] = pr == 0.f ? 0.f : pr * va[e >> 1];
                    z[nt][e & 1] += pr == 0.f ? 0.f : pr * vb[e >> 1];
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t a = pack_bf16(w[2 * h], w[2 * h + 1]);
                    const uint32_t b = pack_bf16(w[2 * h] - __uint_as_float(a << 16), w[2 * h + 1] - __uint_as_float(a & 0xffff0000u));
                    hi[nt][h] = transpose8(a);
                    lo[nt][h] = transpose8(b);
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
                    vw[k][L::kVWords - 1] = u.y;
                } else {
                    vw[k][0] = lds32(stage + L::kCodes + v_chunk<D>(t, r >> 2) + (r & 3) * 4);
                }
            }
#pragma unroll
            for (int w = 0; w < L::kVWords; ++w) {
                const uint32_t a0 = __byte_perm(vw[0][w], vw[1][w], 0x5410), a1 = __byte_perm(vw[0][w], vw[1][w], 0x7632);
                const uint32_t a2 = __byte_perm(vw[2][w], vw[3][w], 0x5410), a3 = __byte_perm(vw[2][w], vw[3][w], 0x7632);
                auto tile = [&](int j, const uint32_t (&a)[4]) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma<true>(o[nt][j], a, hi[nt][0], hi[nt][1]);
                        mma<true>(o[nt][j], a, lo[nt][0], lo[nt][1]);
                    }
                };
                tile(4 * w, {unpack2<true, 0>(a0), unpack2<true, 0>(a1), unpack2<true, 0>(a2), unpack2<true, 0>(a3)});
                tile(4 * w + 1, {unpack2<true, 1>(a0), unpack2<true, 1>(a1), unpack2<true, 1>(a2), unpack2<true, 1>(a3)});
                tile(4 * w + 2, {unpack2<true, 2>(a0), unpack2<true, 2>(a1), unpack2<true, 2>(a2), unpack2<true, 2>(a3)});
                tile(4 * w + 3, {unpack2<true, 3>(a0), unpack2<true, 3>(a1), unpack2<true, 3>(a2), unpack2<true, 3>(a3)});
            }
        }
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
// their running sums through shared memory at the end of a tile.
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

    const Where w = locate(p, blockIdx.x, gridDim.x, scratch);
    if ((long long)blockIdx.x >= w.parts)
        return;
    const long long u0 = w.first, u1 = w.total * (blockIdx.x + 1) / w.parts;
    int b = w.b;
    Span sp = span_of(p, b);
    const int HR = p.Hkv * p.RB;
    int hr = (int)((u0 - w.before) / sp.n);
    int ku = (int)((u0 - w.before) - (long long)hr * sp.n);

    for (long long u = u0; u < u1;) {
        const int ke = (int)((long long)sp.n - ku < u1 - u ? sp.n : ku + (u1 - u));
        const bool whole = ku == 0 && ke == sp.n;
        const int h = hr / p.RB, r0 = (hr - h * p.RB) * (8 * NT);
        const int nrows = p.rows - r0 < 8 * NT ? p.rows - r0 : 8 * NT;
        const long long bh = (long long)b * p.Hkv + h;
        const long long row0 = bh * p.rows + r0;   // of the [B H Nq] query rows

        const int nsub = (ke - ku) * (kUnit / kSub);
        auto token = [&](int s) { return sp.token(ku + s / (kUnit / kSub)) + (s % (kUnit / kSub)) * kSub; };
        // Two stages ahead; the query rows load behind them.
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) {
            const int s = warp + i * kWarps;
            load_stage<D, true>(p, ring + i * L::kStage, bh, s < nsub ? token(s) : 0, sp.len, s < nsub);
        }
        Queries<D, BF16, NT> q;
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
            load_stage<D, true>(p, ring + fill * L::kStage, bh, next < nsub ? token(next) : 0, sp.len, next < nsub);
            const int t0 = token(s);
            a.step(p, ring + st * L::kStage, q, t0, t0 < edge_lo || t0 + kSub > edge_hi, vis);
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
                    jo[n * S::kORow + out_channel<D>(r, j, 0)] = a.o[nt][j][e] + z;
                    jo[n * S::kORow + out_channel<D>(r, j, 1)] = a.o[nt][j][e + 2] + z;
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
        u += ke - ku;
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
    const Where w = locate(p, k + 1, grid, scratch);
    grid_wait();   // by every block, so that this grid ends after the attention has
    const long long G = w.parts, U = w.total;
    if (k + 1 >= G)
        return;
    const long long edge = w.first;   // first unit of CTA k + 1
    const Span sp = span_of(p, w.b);
    const int hr = (int)((edge - w.before) / sp.n);
    const long long t0 = w.before + (long long)hr * sp.n, t1 = t0 + sp.n;   // the tile's units
    if (t0 == edge || U * k / G > t0)   // not inside a tile, or not its first boundary
        return;
    const long long last = (t1 * G - 1) / U;   // CTA holding unit t1 - 1: the largest x with U x / G < t1
    const int h = hr / p.RB, r0 = (hr - h * p.RB) * (8 * NT);
    const int nrows = p.rows - r0 < 8 * NT ? p.rows - r0 : 8 * NT;
    const long long row0 = ((long long)w.b * p.Hkv + h) * p.rows + r0;
    const long long slot0 = 2 * k + (U * k / G == t0 ? 0 : 1);   // CTA k's part: its only one, or its last
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

// acc[b, h, t] (+)= sum over the key head's query rows of exp(x_t - LSE): the
// scores again, K alone, with the LSE that the attention returned.  A token's
// sum is formed by one warp, in a fixed order, and every entry of acc has one
// writer, so nothing is added by atomics.  More than 8 NT query rows go
// through the cache in passes (the later ones read it from L2).
template <int D, bool BF16, int NT>
__global__ void __launch_bounds__(kThreads, NT <= 2 ? 2 : 1) weights_kernel(const Params p)
{
    using L = Layout<D>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long scratch[kWarps + 2];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, r = lane / 4, c = lane % 4;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + (uint32_t)(warp * kStages * L::kKeyStage);
    const Where w = locate(p, blockIdx.x, gridDim.x, scratch);
    if ((long long)blockIdx.x >= w.parts)
        return;
    const long long u0 = w.first, u1 = w.total * (blockIdx.x + 1) / w.parts;
    int b = w.b;
    Span sp = span_of(p, b);
    int h = (int)((u0 - w.before) / sp.n);
    int ku = (int)((u0 - w.before) - (long long)h * sp.n);
    for (long long u = u0; u < u1;) {
        const int ke = (int)((long long)sp.n - ku < u1 - u ? sp.n : ku + (u1 - u));
        const long long bh = (long long)b * p.Hkv + h;
        float *acc = p.acc + bh * p.C;
        const int nsub = (ke - ku) * (kUnit / kSub);
        auto token = [&](int s) { return sp.token(ku + s / (kUnit / kSub)) + (s % (kUnit / kSub)) * kSub; };
        for (int r0 = 0; r0 < p.rows; r0 += 8 * NT) {
            const int nrows = p.rows - r0 < 8 * NT ? p.rows - r0 : 8 * NT;
            const bool add = p.accumulate || r0 > 0;
#pragma unroll
            for (int i = 0; i < kStages - 1; ++i) {
                const int s = warp + i * kWarps;
                load_stage<D, false>(p, ring + i * L::kKeyStage, bh, s < nsub ? token(s) : 0, sp.len, s < nsub);
            }
            Queries<D, BF16, NT> q;
            q.load(p, bh * p.rows + r0, nrows);
            Bounds vis[NT][2];
            float nl[NT][2];   // -LSE in log2 units, -inf for rows that are not there or see nothing
            int edge_lo = 0, edge_hi = 0x7fffffff;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int n = 8 * nt + 2 * c + e;
                    const float lse = n < nrows ? p.lse[bh * p.rows + r0 + n] : -INFINITY;
                    nl[nt][e] = lse == -INFINITY ? -INFINITY : -lse * kLog2e;
                    vis[nt][e] = bounds_of(p, sp.len, r0 + (n < nrows ? n : nrows - 1));
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
                load_stage<D, false>(p, ring + fill * L::kKeyStage, bh, next < nsub ? token(next) : 0, sp.len, next < nsub);
                const int t0 = token(s);
                const bool masked = t0 < edge_lo || t0 + kSub > edge_hi;
                const uint32_t stage = ring + st * L::kKeyStage;
                float sum[4];   // tokens r, r + 8, r + 16, r + 24
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    float x[NT][4];
                    scores<D, BF16, NT>(p, stage, stage + L::kCodes, mt, q, x);
                    sum[2 * mt] = sum[2 * mt + 1] = 0.f;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float y = x[nt][e] + nl[nt][e & 1];
                            const bool hidden = nl[nt][e & 1] == -INFINITY ||
                                                (masked && !sees(vis[nt][e & 1], t0 + 16 * mt + r + 8 * (e >> 1)));
                            sum[2 * mt + (e >> 1)] += hidden ? 0.f : ex2(y);
                        }
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
                    acc[t] = add ? acc[t] + mine : mine;
                st = st + 1 == kStages ? 0 : st + 1;
            }
            cp_wait<0>();
            __syncwarp();
        }
        if (!p.accumulate) {   // entries that no unit holds: between the sinks and the window, and past the sequence
            if (ku == 0)
                for (int t = sp.su * kUnit + threadIdx.x; t < sp.ks * kUnit && t < sp.len; t += kThreads)
                    acc[t] = 0.f;
            if (ke == sp.n)
                for (int t = sp.len + threadIdx.x; t < p.C; t += kThreads)
                    acc[t] = 0.f;
        }
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
