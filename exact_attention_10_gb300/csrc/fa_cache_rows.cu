// fa_cache_rows.cu -- the weights of cached tokens (fa_cache_weights) for more
// than 16 query rows per key head: a prompt's last tokens, or several drafted
// tokens of many query heads.
//
//   acc[b, h, t] (+)= sum over the key head's rows n that see t of
//                     exp(scale q_n . k_t - LSE_n)
//
// With 64 rows the scores are a matrix product of some size (K [tokens, D]
// against Q^T), so they go through the tensor core proper: K's codes, centred
// and exact in fp16 ((code - 7.5) 2^-9, as in fa_cache_kernel.cuh), are
// unpacked into tensor memory, one token to a thread, as the A operand of
// tcgen05.mma, 128 tokens a tile, against up to 64 query rows as B; the scores
// come back from tensor memory as fragments, 16 tokens at a time, two of them
// and a quarter of the columns to a thread, so that a column's constants are
// read for two and a warp's reads of them are few.
//
// What bounds it: issue slots.  Per 128 tokens, 64 rows and D = 128, about 2000
// warp instructions of sums (five per score and thread) and 800 of unpacking,
// 1300 cycles a tile in all, against 256 of the MMAs and 256 of exponentials.
// (With K unpacked into shared memory and one token's scores to a thread it was
// shared memory: 280 cycles of stores, 380 of the MMA's reads and 730 of
// constants of 1400 a tile.  Packed pairs of multiply-adds took as long as
// single ones; 88 registers for the sums and 64 for the unpacking spilled.)
// 2 x 8 key heads, 20000 and 32768 tokens, 64 rows, D = 128: 23.7 us; through
// mma.sync with the rows' fragments in shared memory 30.6.  8 x 8 key heads of
// up to 8192 tokens, D = 128, 18 / 40 / 128 rows: 20.1 / 22.1 / 41.6 us against
// 28.6 / 29.0 / 54.4; 2 x 8 of up to 1024, 18 / 64 rows: 6.9 / 8.0 against 7.1 /
// 7.3, the longer chain of steps.
//
// Roles, beside one another:
//   warps 0-7   the scores' exponentials and sums, two groups of four that take
//               every other tile
//   warps 8-11  unpacking: codes two tiles ahead in registers, fp16 to one of
//               two stages; warp 8 issues the MMAs besides (a warp for that
//               alone would leave the others 72 registers)
// with two CTAs per SM.  Rows are taken 64 at a time; further blocks go
// through the cache again, from L2, and add to what the first wrote.
#include <cuda_runtime.h>

#include "fa_cache_kernel.cuh"
#include "fa_cache_rows.h"
#include "fa_fwd_kernel.cuh"
#include "fa_host.h"

namespace fa {
namespace cache {

namespace {

constexpr int kRowBlock = 64;       // query rows per pass over the cache
constexpr int kTileTokens = 128;    // tokens per MMA tile: two units
constexpr int kRowsThreads = 384;
constexpr int kUnpackWarp = 8;      // the first of the four, which also issues the MMAs
constexpr int kScoreCols = 2 * kRowBlock;   // TMEM: two stages of scores, then two of K (D / 2 columns each)
constexpr uint32_t kTmemCols = 256;         // (two CTAs per SM share 512)

// Wait sites for the status word.
enum : uint32_t { kSiteRowsQueries = 64, kSiteRowsFull, kSiteRowsFree, kSiteRowsDone, kSiteRowsReuse, kSiteRowsDrain };

template <int D>
struct RowsSmem {
    static constexpr int kBoxes = D / 64;                        // 64 channels: a 128-byte swizzled row
    static constexpr int kQBox = kRowBlock * 128;
    static constexpr int kConstOff = kBoxes * kQBox;             // the rows' constants, see load_rows
    static constexpr int kBoundsOff = kConstOff + 4 * kRowBlock * 4;
    static constexpr int kEdgeOff = kBoundsOff + kRowBlock * 16;
    static constexpr int kBarOff = kEdgeOff + 2 * kWarps * 4;
    static constexpr int kScratchOff = kBarOff + 8 * 8;
    static constexpr int kMiscOff = kScratchOff + (kWarps + 2) * 8;
    static constexpr int kBytes = kMiscOff + 16 + 1024;          // (1024: alignment of the swizzle)
};

struct RowsBars {
    uint32_t base;
    __device__ uint32_t full(int s) const { return base + 8u * s; }         // unpacking -> MMA: stage s of K holds a tile
    __device__ uint32_t done(int s) const { return base + 8u * (2 + s); }   // MMA: K s read, scores s final
    __device__ uint32_t free_(int s) const { return base + 8u * (4 + s); }  // sums -> MMA: scores s read out
    __device__ uint32_t rows() const { return base + 8u * 7; }              // queries -> MMA: the block of rows is there
    __device__ uint32_t drain() const { return base + 8u * 6; }
};

// The 32 tokens of tile i of a segment (units [ku, ke)) that a warp of quadrant
// `quad` has: t0 .., of which those before `end` are there.
__device__ __forceinline__ int tile_tokens(const Span &sp, int ku, int ke, int i, int quad, int &end)
{
    const int u = ku + 2 * i + quad / 2;
    end = u < ke ? sp.len : 0;
    return sp.token(u) + quad % 2 * kSub;
}

// Loads that stay where they are written: ahead of their use.
__device__ __forceinline__ uint4 ld_ahead(const uint4 *p)
{
    uint4 v;
    asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

__device__ __forceinline__ uint32_t ld_ahead(const uint32_t *p)
{
    uint32_t v;
    asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

// Row `row` of the query block, 16-byte chunk `ch` of its fp16 values: 8
// channels, in the order in which K's come out of a word of codes, the pairs
// (0, 4), (1, 5), (2, 6), (3, 7).
__device__ __forceinline__ uint32_t chunk_at(uint32_t box0, uint32_t box_bytes, int row, int ch)
{
    return box0 + (uint32_t)(ch / 8) * box_bytes + (uint32_t)row * 128u + (uint32_t)(((ch & 7) ^ (row & 7)) * 16);
}

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// Rows 8 warp + r of the query block (r = lane / 4; channels [c D/4, (c + 1)
// D/4) of lane c): fp16 times a power of two, as Queries::load does it, and
// the row's constants and bounds.  Rows that are not there weigh nothing.  The
// constants of rows 2 i and 2 i + 1 are eight floats: mul, sum, -ref, rest of both.
template <int D, bool BF16>
__device__ __forceinline__ void load_rows(const Params &p, long long bh, int r0, int len, uint32_t base, uint8_t *base_ptr)
{
    using S = RowsSmem<D>;
    constexpr int kWords = D / 32;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, r = lane / 4, c = lane % 4;
    const int n = 8 * warp + r;
    const bool there = r0 + n < p.rows;
    const float lse = there ? __uint_as_float(ld_ahead(reinterpret_cast<const uint32_t *>(p.lse) + bh * p.rows + r0 + n)) : -INFINITY;
    float x[kWords][8], s = 0.f, mx = 0.f;
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (there)
            v = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint32_t *>(p.q) + (bh * p.rows + r0 + n) * (D / 2)) +
                      c * kWords + w);
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
    int e = mx > 0.f ? 14 - (int)((__float_as_uint(mx) >> 23) & 255u) + 127 : 0;
    e = e > 100 ? 100 : (e < -100 ? -100 : e);
    const float up = exp2i(e);
#pragma unroll
    for (int w = 0; w < kWords; ++w)
        sts128(chunk_at(base, S::kQBox, n, c * kWords + w), pack_f16(x[w][0] * up, x[w][4] * up),
               pack_f16(x[w][1] * up, x[w][5] * up), pack_f16(x[w][2] * up, x[w][6] * up),
               pack_f16(x[w][3] * up, x[w][7] * up));
    int lo = 0, hi = 0x7fffffff;
    if (c == 0) {
        const float ref = lse * kLog2e;
        float *k = reinterpret_cast<float *>(base_ptr + S::kConstOff) + n / 2 * 8 + n % 2;
        k[0] = p.qk2 * exp2i(9 - e);
        k[2] = s * p.qk2;
        // what the scores are taken relative to; -inf where the row is not there or sees nothing
        k[4] = lse == -INFINITY ? -INFINITY : -ref;
        // 2 to the power of what its rounding left out
        k[6] = lse == -INFINITY ? 1.f : exp2f(-fmaf(lse, kLog2e, -ref) - lse * kLog2eRest);
        const Bounds v = bounds_of(p, len, there ? r0 + n : p.rows - 1);
        reinterpret_cast<int4 *>(base_ptr + S::kBoundsOff)[n] = make_int4(v.lo, v.hi, v.sink, 0);
        lo = v.lo;
        hi = v.hi;
    }
    lo = __reduce_max_sync(0xffffffffu, lo);
    hi = __reduce_min_sync(0xffffffffu, hi);
    if (lane == 0) {
        int *edge = reinterpret_cast<int *>(base_ptr + S::kEdgeOff);
        edge[warp] = lo;
        edge[kWarps + warp] = hi;
    }
}

// Unpacking: a thread has one token of the tile (its TMEM lane), whose codes it
// loads two tiles ahead.
template <int D>
struct Unpacker {
    static constexpr int kChunks = D / 32;   // of 16 bytes, codes of a token
    uint4 next[2][kChunks];

    __device__ __forceinline__ void fetch(uint4 (&x)[kChunks], const uint8_t *kc, const Span &sp, int ku, int ke, int i)
    {
        int end;
        const int t = tile_tokens(sp, ku, ke, i, threadIdx.x / 32 % 4, end) + threadIdx.x % 32;
        const uint4 *src = reinterpret_cast<const uint4 *>(kc + (long long)t * (D / 2));
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            x[k] = make_uint4(0u, 0u, 0u, 0u);
            if (t < end)
                x[k] = ld_ahead(src + k);
        }
    }

    // fp16 pairs, 16 columns per chunk, to `stage` (the warp's lanes).
    __device__ __forceinline__ void store(const uint4 (&x)[kChunks], uint32_t stage)
    {
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
            uint32_t v[16];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[4 * j] = centred_even(w[j]);
                v[4 * j + 1] = centred_odd(w[j]);
                v[4 * j + 2] = centred_even(w[j] >> 8);
                v[4 * j + 3] = centred_odd(w[j] >> 8);
            }
            ptx::tmem_st16(stage + 16 * k, v);
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before_sync();
    }
};

// Adds to the sums of two tokens (t and t + 8) this thread's columns, two of
// each eight, of x, whose first column's constants and bounds are at k and vis.
template <int N, bool MASKED>
__device__ __forceinline__ void add_columns(const uint32_t (&x)[N], int cols, const float *k, const int4 *vis, int t,
                                            const float (&sa)[2], const float (&za)[2], float (&sum)[2])
{
#pragma unroll
    for (int q = 0; q < N / 4; ++q) {
        if (q % 2 == 0 && 8 * q >= cols)
            break;
        const float4 a = *reinterpret_cast<const float4 *>(k + 32 * q);       // mul, sum
        const float4 b = *reinterpret_cast<const float4 *>(k + 32 * q + 4);   // -ref, rest
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float y0 = fmaf(__uint_as_float(x[4 * q + 2 * j]) * a.x, sa[j], fmaf(za[j], a.z, b.x));
            float y1 = fmaf(__uint_as_float(x[4 * q + 2 * j + 1]) * a.y, sa[j], fmaf(za[j], a.w, b.y));
            if (MASKED) {
                const int4 v0 = vis[8 * q], v1 = vis[8 * q + 1];
                y0 = sees(Bounds{v0.x, v0.y, v0.z}, t + 8 * j) ? y0 : -INFINITY;
                y1 = sees(Bounds{v1.x, v1.y, v1.z}, t + 8 * j) ? y1 : -INFINITY;
            }
            sum[j] = fmaf(ex2(y0), b.z, sum[j]);
            sum[j] = fmaf(ex2(y1), b.w, sum[j]);
        }
    }
}

// The sums of a warp's 32 tokens from t0 on, over `cols` columns (at most 2 W)
// of scores at `at`: total[j] of token t0 + lane / 4 + 8 j.  The next 16 tokens'
// or columns' scores load while these are worked on; `bar` is arrived on once
// all have been read.
template <bool BF16, int W, bool MASKED>
__device__ __forceinline__ void tile_sums(uint32_t at, int cols, uint32_t par, const float *k, const int4 *vis, int t0,
                                          uint32_t bar, float (&total)[4])
{
    const int lane = threadIdx.x % 32, r = lane / 4, cl = lane % 4;
    k += 8 * cl;
    vis += 2 * cl;
    uint32_t x[W / 2], y[W / 2];
    ptx::tmem_ld_frag(at, x);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        float sa[2], za[2], sum[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t v = __shfl_sync(0xffffffffu, par, r + 16 * half + 8 * j);
            const float a = to_float<BF16>(v & 0xffffu), z = fmaf(7.5f, a, to_float<BF16>(v >> 16));
            sa[j] = a;
            za[j] = z;
        }
        const int t = t0 + 16 * half + r;
        ptx::tmem_wait_ld();
        ptx::tmem_ld_frag(at + (half << 20) + W, y);
        add_columns<W / 2, MASKED>(x, W, k, vis, t, sa, za, sum);
        ptx::tmem_wait_ld();
        if (half == 0) {
            ptx::tmem_ld_frag(at + (1u << 20), x);
        } else {
            ptx::tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                ptx::mbar_arrive(bar);
        }
        add_columns<W / 2, MASKED>(y, cols - W, k + 4 * W, vis + W, t, sa, za, sum);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float a = sum[j];
            a += __shfl_xor_sync(0xffffffffu, a, 1);
            total[2 * half + j] = a + __shfl_xor_sync(0xffffffffu, a, 2);
        }
    }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kRowsThreads, 2) weights_rows_kernel(const Params p)
{
    using S = RowsSmem<D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *base_ptr = smem_raw + (base - raw);
    const RowsBars b{base + S::kBarOff};
    uint32_t *misc = reinterpret_cast<uint32_t *>(base_ptr + S::kMiscOff);
    const Ctl c{reinterpret_cast<volatile int *>(misc + 1)};
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    const Where w = locate_quick(p, blockIdx.x, gridDim.x, reinterpret_cast<long long *>(base_ptr + S::kScratchOff));
    if ((long long)blockIdx.x >= w.parts)
        return;
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(b.full(s), 4);
            ptx::mbar_init(b.done(s), 1);
            ptx::mbar_init(b.free_(s), 4);
        }
        ptx::mbar_init(b.rows(), kWarps);
        ptx::mbar_init(b.drain(), 1);
        *c.abort_flag = 0;
        ptx::fence_barrier_init();
    }
    if (warp == kUnpackWarp) {
        ptx::tmem_alloc(ptx::smem_addr(misc), kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(misc);

    const long long u0 = w.first, u1 = share_of(w, blockIdx.x + 1);
    int bb = w.b;
    Span sp = span_of(p, bb);
    int h = tile_of(u0 - w.before, sp.n);
    int ku = (int)((u0 - w.before) - (long long)h * sp.n);
    uint32_t it = 0;   // tiles before this pass: tile j of it is number it + j, in stage (it + j) % 2
    uint32_t pass = 0;
    bool ok = true;
    for (long long u = u0; u < u1 && ok;) {
        const int ke = (int)((long long)sp.n - ku < u1 - u ? sp.n : ku + (u1 - u));
        const long long bh = (long long)bb * p.Hkv + h;
        float *acc = p.acc + bh * p.C;
        const int nt = (ke - ku + 1) / 2;
        for (int r0 = 0; r0 < p.rows && ok; r0 += kRowBlock) {
            const int nrows = p.rows - r0 < kRowBlock ? p.rows - r0 : kRowBlock;
            const int cols = (nrows + 15) & ~15;
            // Every role is through with the block before.  The sums' warps bring
            // the next rows while the others unpack the first tiles.
            if (warp < kWarps) {
                load_rows<D, BF16>(p, bh, r0, sp.len, base, base_ptr);
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    ptx::mbar_arrive(b.rows());
                asm volatile("bar.sync 1, 256;" ::: "memory");   // the sums' warps have the constants
            }
            if (warp >= kUnpackWarp) {
                const uint32_t idesc = instr_desc_f16(false, kTileTokens, cols, false);
                Unpacker<D> x;
                const uint8_t *kc = p.kc + bh * p.C * (D / 2);
                x.fetch(x.next[0], kc, sp, ku, ke, 0);
                x.fetch(x.next[1], kc, sp, ku, ke, 1);
                for (int i = 0; i < nt && ok; i += 2) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t n = it + i + e, s = n & 1u;
                        const uint32_t k_at = tmem + kScoreCols + s * (D / 2);
                        if (i + e >= nt)
                            break;
                        if (n >= 2 && !warp_wait(b.done(s), ((n >> 1) - 1u) & 1u, c, kSiteRowsReuse)) {
                            ok = false;
                            break;
                        }
                        ptx::tc_fence_after_sync();
                        x.store(x.next[e], k_at + ((uint32_t)(warp % 4) << 21));
                        __syncwarp();
                        if (lane == 0)
                            ptx::mbar_arrive(b.full(s));
                        x.fetch(x.next[e], kc, sp, ku, ke, i + e + 2);
                        if (warp > kUnpackWarp)
                            continue;
                        if (i + e == 0 && !(ok = warp_wait(b.rows(), pass & 1u, c, kSiteRowsQueries)))
                            break;
                        ok = warp_wait(b.full(s), (n >> 1) & 1u, c, kSiteRowsFull) &&
                             (n < 2 || warp_wait(b.free_(s), ((n >> 1) - 1u) & 1u, c, kSiteRowsFree));
                        if (!ok)
                            break;
                        ptx::tc_fence_after_sync();
                        if (ptx::elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk)
                                ptx::mma_ts(tmem + s * kRowBlock, k_at + kk * 8,
                                            smem_desc_sw128(base + (kk / 4) * S::kQBox + (kk % 4) * 32, 16), idesc,
                                            kk > 0 ? 1u : 0u);
                            ptx::mma_commit(b.done(s));
                        }
                        __syncwarp();
                    }
                }
            } else {
                const bool add = p.accumulate || r0 > 0;
                const float *k = reinterpret_cast<const float *>(base_ptr + S::kConstOff);
                const int4 *bounds = reinterpret_cast<const int4 *>(base_ptr + S::kBoundsOff);
                const int *edge = reinterpret_cast<const int *>(base_ptr + S::kEdgeOff);
                int edge_lo = 0, edge_hi = 0x7fffffff;
#pragma unroll
                for (int i = 0; i < kWarps; ++i) {
                    edge_lo = max(edge_lo, edge[i]);
                    edge_hi = min(edge_hi, edge[kWarps + i]);
                }
                const uint32_t *kp = p.kp + bh * p.C;
                const int g = warp / 4, quad = warp % 4;   // of the two groups: the tiles of stage g
                const int r = lane / 4, cl = lane % 4;
                const uint32_t scores_at = tmem + g * kRowBlock + ((uint32_t)quad << 21);
                const int first = (int)((g ^ it) & 1u);
                int end, t0 = tile_tokens(sp, ku, ke, first, quad, end);
                uint32_t par = t0 + lane < end ? ld_ahead(kp + t0 + lane) : 0u;
                for (int i = first; i < nt; i += 2) {
                    const uint32_t n = it + i, now = par;
                    const int t = t0;
                    // lane (r, cl) writes token r + 8 cl
                    float *to = t + r + 8 * cl < end ? acc + t + r + 8 * cl : nullptr;
                    const float old = add && to ? *to : 0.f;
                    t0 = tile_tokens(sp, ku, ke, i + 2, quad, end);
                    par = t0 + lane < end ? ld_ahead(kp + t0 + lane) : 0u;
                    if (!warp_wait(b.done(g), (n >> 1) & 1u, c, kSiteRowsDone)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after_sync();
                    const bool masked = t < edge_lo || t + kSub > edge_hi;
                    float total[4];
                    if (cols > 32) {
                        if (masked)
                            tile_sums<BF16, 32, true>(scores_at, cols, now, k, bounds, t, b.free_(g), total);
                        else
                            tile_sums<BF16, 32, false>(scores_at, cols, now, k, bounds, t, b.free_(g), total);
                    } else {
                        if (masked)
                            tile_sums<BF16, 16, true>(scores_at, cols, now, k, bounds, t, b.free_(g), total);
                        else
                            tile_sums<BF16, 16, false>(scores_at, cols, now, k, bounds, t, b.free_(g), total);
                    }
                    if (to)
                        *to = old + (cl == 0 ? total[0] : (cl == 1 ? total[1] : (cl == 2 ? total[2] : total[3])));
                }
            }
            ++pass;
            it += (uint32_t)nt;
            ok = __syncthreads_and(ok);
        }
        if (!p.accumulate && warp < kWarps)
            zero_rest(p, acc, sp, ku, ke);
        u += ke - ku;
        ku = 0;
        if (++h == p.Hkv && u < u1) {
            h = 0;
            sp = span_of(p, ++bb);
        }
    }
    if (warp == kUnpackWarp) {   // every MMA has completed before its TMEM is given back
        if (ptx::elect_one())
            ptx::mma_commit(b.drain());
        __syncwarp();
        wait_landed(b.drain(), 0u, c, kSiteRowsDrain);
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    if (warp == kUnpackWarp) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D, bool BF16>
fa_status launch(const Params &p, int sms, cudaStream_t s, int dev)
{
    constexpr int smem = RowsSmem<D>::kBytes;
    static bool set[fa_host::kMaxDevices] = {};
    const fa_status st = fa_host::allow_smem(reinterpret_cast<const void *>(&weights_rows_kernel<D, BF16>), smem, dev, set);
    if (st != FA_OK)
        return st;
    weights_rows_kernel<D, BF16><<<sms * 2, kRowsThreads, smem, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace

}  // namespace cache
}  // namespace fa

namespace fa_launch {

fa_status launch_weights_rows(const fa::cache::Params &p, int D, bool bf16, int sms, cudaStream_t s, int dev)
{
    if (D == 64)
        return bf16 ? fa::cache::launch<64, true>(p, sms, s, dev) : fa::cache::launch<64, false>(p, sms, s, dev);
    return bf16 ? fa::cache::launch<128, true>(p, sms, s, dev) : fa::cache::launch<128, false>(p, sms, s, dev);
}

unsigned int *status_word_rows()
{
    return fa::status_word_address();
}

}  // namespace fa_launch
