// coli_adapters.cuh -- low-rank adapters of many requests in one batch
// (coli_adapters_forward), added beside a projection that all requests share:
//   out_t = base_t + scale_a B_a (A_a x_t),  a = the adapter of token t
// A_a is [rank, K], B_a is [N, rank], bf16; tokens without an adapter keep base.
//
// Tokens are grouped into tiles of up to 32 of one adapter, so each adapter is
// read once per tile.  Two kernels:
//   shrink   h = A_a x for (tile, piece of K): eight warps take 32-K blocks,
//            their sums meet in shared memory, one fp32 partial row per piece
//   expand   out for (tile, columns): the pieces of h are summed in order, scaled,
//            cut into bf16 parts; each warp multiplies them with 32 rows of B_a at
//            a time and adds base
// Memory-bound: at 4096 tokens, K = N = 6144, rank 64 the arithmetic is 6.4 GFLOP
// against 176 MB, 4 us of tensor work beside 27 us of traffic, so the products run
// on warp-level mma (m16n8k16, fp32 accumulation) whose operands come straight
// from global memory: K (and the rank) may be summed in any order, so lane q of a
// quad takes 8 consecutive values of each 32, one 16-byte load that serves two
// MMAs, and the output columns are dealt so that a lane ends with 8 consecutive
// ones.  No staging of x, A or B.
//
// fp32 activations enter as three exact bf16 parts.  h is cut into three parts
// for fp32 outputs (exact) and two for bf16 outputs (8 bits cut, 8 rounded: 2^-16
// of h, against the output's own rounding of 2^-9).
#pragma once

#include "coli_common.cuh"

namespace coli {

constexpr int kLoTile = 32;      // tokens per tile
constexpr int kLoThreads = 256;
constexpr int kLoWarps = kLoThreads / 32;
constexpr int kLoMaxRank = 256;
constexpr int kLoRB = 64;        // rank values accumulated at a time in the shrink kernel
constexpr int kLoSmallT = 64;    // batches up to this size are grouped inside each block
constexpr int kLoGroupThreads = 1024;

struct LoArgs {
    int T, K, N, R, n;       // R: row length of the stored adapters; n adapters
    const void* x;           // [T, K]
    const uint16_t* a;       // [n, R, K]
    const uint16_t* b;       // [n, N, R]
    const int32_t* rank;     // [n] or null: all R
    const float* scale;      // [n]
    const int32_t* which;    // [T] adapter of each token
    const void* base;        // [T, N] or null
    void* out;               // [T, N]
    float* h;                // [pieces, T, R]
    int pieces, chunk;       // pieces of K, chunk values each (a multiple of 32)
    int cols;                // columns per block of the expand kernel (a multiple of 32)
    int32_t* perm;           // [T] tokens by adapter (large batches)
    int32_t* tiles;          // [3 max_tiles] adapter, first position, count
    int32_t* n_tiles;        // [1]
    int max_tiles;
};

// The adapter of a token; anything outside [0, n) is none (n).
__device__ __forceinline__ int lo_adapter(const LoArgs& a, int t)
{
    const int w = a.which[t];
    return w >= 0 && w < a.n ? w : a.n;
}

// Tokens by adapter for large batches: a counting sort by one block (n + 1 bins,
// the last for tokens without an adapter) and the table of tiles.  A warp adds
// each distinct adapter of its 32 tokens once.  The order inside an adapter does
// not matter to any result: every token's sums are its own.
__global__ void __launch_bounds__(kLoGroupThreads) lo_group_kernel(const __grid_constant__ LoArgs a)
{
    __shared__ int count[kMaxExperts + 1], first[kMaxExperts + 1], tile0[kMaxExperts + 1];
    __shared__ int wsum[2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, bins = a.n + 1;
    for (int i = threadIdx.x; i < bins; i += kLoGroupThreads) count[i] = 0;
    __syncthreads();
    griddep_launch_dependents();
    for (int t0 = warp * 32; t0 < a.T; t0 += kLoGroupThreads) {
        const int t = t0 + lane;
        const int w = t < a.T ? lo_adapter(a, t) : -1;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, w);
        if (w >= 0 && lane == __ffs(same) - 1) atomicAdd(&count[w], __popc(same));
    }
    __syncthreads();
    // exclusive sums of tokens and tiles over the bins, 1024 at a time
    int base_c = 0, base_t = 0;
    for (int b0 = 0; b0 < bins; b0 += kLoGroupThreads) {
        const int b = b0 + threadIdx.x;
        const int c = b < bins ? count[b] : 0, nt = (c + kLoTile - 1) / kLoTile;
        int ic = c, it = nt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int yc = __shfl_up_sync(0xFFFFFFFFu, ic, o), yt = __shfl_up_sync(0xFFFFFFFFu, it, o);
            if (lane >= o) ic += yc, it += yt;
        }
        if (lane == 31) wsum[0][warp] = ic, wsum[1][warp] = it;
        __syncthreads();
        int pc = 0, pt = 0, all_c = 0, all_t = 0;
        for (int w = 0; w < kLoGroupThreads / 32; ++w) {
            if (w == warp) pc = all_c, pt = all_t;
            all_c += wsum[0][w], all_t += wsum[1][w];
        }
        if (b < bins) {
            first[b] = base_c + pc + ic - c;
            tile0[b] = base_t + pt + it - nt;
            for (int i = 0; i < nt; ++i) {
                int32_t* e = a.tiles + 3 * (tile0[b] + i);
                e[0] = b;
                e[1] = first[b] + i * kLoTile;
                e[2] = min(kLoTile, c - i * kLoTile);
            }
        }
        base_c += all_c, base_t += all_t;
        __syncthreads();
    }
    if (threadIdx.x == 0) *a.n_tiles = base_t;
    for (int t0 = warp * 32; t0 < a.T; t0 += kLoGroupThreads) {
        const int t = t0 + lane;
        const int w = t < a.T ? lo_adapter(a, t) : -1;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, w);
        const int leader = __ffs(same) - 1;
        int at = 0;
        if (w >= 0 && lane == leader) at = atomicAdd(&first[w], __popc(same));
        at = __shfl_sync(0xFFFFFFFFu, at, leader) + __popc(same & ((1u << lane) - 1u));
        if (w >= 0) a.perm[at] = t;
    }
}

// The tile of a block: its adapter and tokens.  Shared memory of the two kernels.
struct LoTile {
    int adapter, count;
    int token[kLoTile];
    int of[kLoSmallT], start[kLoSmallT];  // grouping of a small batch
};

// Fills `s` for tile number `tile`; false when there is no such tile.  Small
// batches are grouped here, by first token of each adapter; large ones were
// grouped by lo_group_kernel.  All threads call it.
__device__ __forceinline__ bool lo_find_tile(const LoArgs& a, int tile, LoTile& s)
{
    const int tid = threadIdx.x;
    if (a.T > kLoSmallT) {
        if (tile >= *a.n_tiles) return false;
        const int32_t* e = a.tiles + 3 * tile;
        if (tid == 0) s.adapter = e[0], s.count = e[2];
        if (tid < kLoTile) s.token[tid] = a.perm[e[1] + min(tid, e[2] - 1)];  // the tail repeats a token
        __syncthreads();
        return true;
    }
    if (tid == 0) s.count = 0;
    int w = -1;
    if (tid < kLoSmallT) s.of[tid] = w = tid < a.T ? lo_adapter(a, tid) : -1;
    __syncthreads();
    int cnt = 0, pos = 0, lead = 0;
    if (tid < a.T) {
        for (int i = a.T - 1; i >= 0; --i) {
            const bool same = s.of[i] == w;
            cnt += same ? 1 : 0;
            pos += same && i < tid ? 1 : 0;
            if (same) lead = i;
        }
        s.start[tid] = pos == 0 ? (cnt + kLoTile - 1) / kLoTile : 0;
    }
    __syncthreads();
    if (tid < a.T) {
        int t0 = 0;  // first tile of this token's adapter
        for (int i = 0; i < lead; ++i) t0 += s.start[i];
        if (t0 + pos / kLoTile == tile) {
            s.token[pos % kLoTile] = tid;
            if (pos % kLoTile == 0) {
                s.adapter = w;
                s.count = min(kLoTile, cnt - pos);
            }
        }
    }
    __syncthreads();
    const int c = s.count;
    if (c == 0) return false;
    if (tid >= c && tid < kLoTile) s.token[tid] = s.token[0];
    __syncthreads();
    return true;
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Top 16 bits of two floats as a bf16 pair; the rest of each stays in lo, hi (exact).
__device__ __forceinline__ uint32_t cut_pair(float& lo, float& hi)
{
    const uint32_t w = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
    lo -= __uint_as_float(w << 16);
    hi -= __uint_as_float(w & 0xFFFF0000u);
    return w;
}

// h[t, r] of one piece of K.  Grid (tiles, pieces).
template <bool kX16>
__global__ void __launch_bounds__(kLoThreads) lo_shrink_kernel(const __grid_constant__ LoArgs a)
{
    constexpr int kParts = kX16 ? 1 : 3;
    __shared__ LoTile s;
    __shared__ __align__(16) float sum[kLoWarps / 2][kLoTile * kLoRB];
    griddep_wait();
    griddep_launch_dependents();
    if (!lo_find_tile(a, blockIdx.x, s) || s.adapter == a.n) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int ad = s.adapter, rank = a.rank ? min(max(a.rank[ad], 0), a.R) : a.R;
    const bool two = s.count > 16;  // a second 16-row half
    const int k0 = blockIdx.y * a.chunk, k1 = min(a.K, k0 + a.chunk);
    const size_t es = kX16 ? 2 : 4;
    const char* xr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) xr[i] = static_cast<const char*>(a.x) + ((size_t)s.token[g + 8 * i] * a.K + 8 * q) * es;
    for (int r0 = 0; r0 < rank; r0 += kLoRB) {
        const int nt = min(kLoRB / 8, (rank - r0 + 7) / 8);
        const uint16_t* ap = a.a + ((size_t)ad * a.R + r0 + g) * a.K + 8 * q;
        float acc[2][kLoRB / 8][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int j = 0; j < kLoRB / 8; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[m][j][c] = 0.f;
#pragma unroll 1
        for (int k = k0 + 32 * warp; k < k1; k += 32 * kLoWarps) {
            const bool in = k + 8 * q < a.K;  // K is a multiple of 8: whole lanes end
            uint4 w[kLoRB / 8];
#pragma unroll
            for (int j = 0; j < kLoRB / 8; ++j) {
                w[j] = make_uint4(0u, 0u, 0u, 0u);
                if (in && j < nt && r0 + 8 * j + g < rank) w[j] = *reinterpret_cast<const uint4*>(ap + (size_t)8 * j * a.K + k);
            }
            uint4 xv[4][kX16 ? 1 : 2];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int v = 0; v < (kX16 ? 1 : 2); ++v) {
                    xv[i][v] = make_uint4(0u, 0u, 0u, 0u);
                    if (in && (i < 2 || two)) xv[i][v] = *reinterpret_cast<const uint4*>(xr[i] + (size_t)k * es + 16 * v);
                }
            // parts of x: four bf16 pairs per row and part, pairs 0, 1 for the first MMA, 2, 3 for the second
            uint32_t p[kParts][4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (kX16) {
                    p[0][i][0] = xv[i][0].x, p[0][i][1] = xv[i][0].y, p[0][i][2] = xv[i][0].z, p[0][i][3] = xv[i][0].w;
                } else {
                    float f[8] = {__uint_as_float(xv[i][0].x), __uint_as_float(xv[i][0].y), __uint_as_float(xv[i][0].z),
                                  __uint_as_float(xv[i][0].w), __uint_as_float(xv[i][1].x), __uint_as_float(xv[i][1].y),
                                  __uint_as_float(xv[i][1].z), __uint_as_float(xv[i][1].w)};
#pragma unroll
                    for (int u = 0; u < kParts; ++u)
#pragma unroll
                        for (int c = 0; c < 4; ++c) p[u][i][c] = cut_pair(f[2 * c], f[2 * c + 1]);
                }
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                if (m == 1 && !two) break;
#pragma unroll
                for (int j = 0; j < kLoRB / 8; ++j) {
                    if (j >= nt) break;
#pragma unroll
                    for (int u = kParts - 1; u >= 0; --u) {  // small parts first
                        mma_bf16(acc[m][j], p[u][2 * m][0], p[u][2 * m + 1][0], p[u][2 * m][1], p[u][2 * m + 1][1], w[j].x, w[j].y);
                        mma_bf16(acc[m][j], p[u][2 * m][2], p[u][2 * m + 1][2], p[u][2 * m][3], p[u][2 * m + 1][3], w[j].z, w[j].w);
                    }
                }
            }
        }
        // sum of the warps: the upper half hands its sums to the lower, three times
#pragma unroll
        for (int half = kLoWarps / 2; half > 0; half >>= 1) {
            __syncthreads();
            if (warp >= half && warp < 2 * half) {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int j = 0; j < kLoRB / 8; ++j)
                        if (j < nt && (m == 0 || two))
                            *reinterpret_cast<float4*>(&sum[warp - half][((m * (kLoRB / 8) + j) * 32 + lane) * 4]) =
                                make_float4(acc[m][j][0], acc[m][j][1], acc[m][j][2], acc[m][j][3]);
            }
            __syncthreads();
            if (warp < half) {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int j = 0; j < kLoRB / 8; ++j)
                        if (j < nt && (m == 0 || two)) {
                            const float4 o =
                                *reinterpret_cast<const float4*>(&sum[warp][((m * (kLoRB / 8) + j) * 32 + lane) * 4]);
                            acc[m][j][0] += o.x, acc[m][j][1] += o.y, acc[m][j][2] += o.z, acc[m][j][3] += o.w;
                        }
            }
        }
        if (warp == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (g + 8 * i >= s.count) continue;
                float* hp = a.h + ((size_t)blockIdx.y * a.T + s.token[g + 8 * i]) * a.R + r0 + 2 * q;
#pragma unroll
                for (int j = 0; j < kLoRB / 8; ++j)
                    if (j < nt) {
                        const float* c = &acc[i >> 1][j][(i & 1) * 2];
                        *reinterpret_cast<float2*>(hp + 8 * j) = make_float2(c[0], c[1]);
                    }
            }
        }
    }
}

// out = base + (scale h) B^T for a tile and `cols` columns.  Grid (tiles, column blocks).
// Shared memory: the parts of scale h, [kParts][32][rs] bf16, rs = R rounded to 32, + 8 (rows on other banks).
template <bool kO16>
__global__ void __launch_bounds__(kLoThreads) lo_expand_kernel(const __grid_constant__ LoArgs a)
{
    constexpr int kParts = kO16 ? 2 : 3;
    extern __shared__ __align__(16) uint16_t hs[];
    __shared__ LoTile s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    griddep_wait();
    if (!lo_find_tile(a, blockIdx.x, s)) return;
    const int ad = s.adapter;
    if (ad == a.n && a.base == a.out) return;  // in place: nothing to add
    const int rank = ad == a.n ? 0 : a.rank ? min(max(a.rank[ad], 0), a.R) : a.R;
    const int rp = (rank + 31) / 32 * 32, rs = (a.R + 31) / 32 * 32 + 8;
    const bool two = s.count > 16;
    if (rank > 0) {
        const float scale = a.scale[ad];
        const size_t plane = (size_t)a.T * a.R;
        for (int i = threadIdx.x; i < kLoTile * (rp / 2); i += kLoThreads) {
            const int row = i / (rp / 2), r = 2 * (i - row * (rp / 2));
            float v0 = 0.f, v1 = 0.f;
            if (row < s.count && r < rank) {  // R is even, so a pair is inside the row
                const float* hp = a.h + (size_t)s.token[row] * a.R + r;
                for (int p = 0; p < a.pieces; ++p) {
                    const float2 o = *reinterpret_cast<const float2*>(hp + p * plane);
                    v0 += o.x, v1 += o.y;
                }
                v0 *= scale;
                v1 = r + 1 < rank ? v1 * scale : 0.f;
            }
#pragma unroll
            for (int u = 0; u < kParts; ++u) {
                uint32_t w;
                if (kO16 && u == kParts - 1) {  // the last of two parts is rounded, not cut
                    const __nv_bfloat162 v = __floats2bfloat162_rn(v0, v1);
                    w = *reinterpret_cast<const uint32_t*>(&v);
                } else {
                    w = cut_pair(v0, v1);
                }
                *reinterpret_cast<uint32_t*>(hs + (size_t)(u * kLoTile + row) * rs + r) = w;
            }
        }
        __syncthreads();
    }
    const int c_end = min(a.N, (int)(blockIdx.y + 1) * a.cols);
    for (int n0 = blockIdx.y * a.cols + 32 * warp; n0 < c_end; n0 += 32 * kLoWarps) {
        const int col = n0 + 8 * q;  // this lane's 8 columns (N is a multiple of 8)
        const bool cin = col < a.N;
        // base first: its loads are under way while the products run
        uint4 bv[4][kO16 ? 1 : 2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int v = 0; v < (kO16 ? 1 : 2); ++v) {
                bv[i][v] = make_uint4(0u, 0u, 0u, 0u);
                if (a.base && cin && g + 8 * i < s.count)
                    bv[i][v] = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.base) +
                                                               ((size_t)s.token[g + 8 * i] * a.N + col) * (kO16 ? 2 : 4) + 16 * v);
            }
        float acc[2][4][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[m][j][c] = 0.f;
        // column g of MMA j is output column n0 + 8 (g / 2) + 2 j + g % 2: lane q's results are 8 q + 0..7
        const int brow = n0 + 8 * (g >> 1) + (g & 1);
        for (int r = 0; r < rank; r += 32) {
            uint4 w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[j] = make_uint4(0u, 0u, 0u, 0u);
                const int rr = r + 8 * q;
                if (brow + 2 * j < a.N && rr < rank) {
                    w[j] = *reinterpret_cast<const uint4*>(a.b + ((size_t)ad * a.N + brow + 2 * j) * a.R + rr);
                    if (rr + 8 > rank) {  // what lies behind the adapter's rank does not count, whatever it is
                        uint32_t* e = reinterpret_cast<uint32_t*>(&w[j]);
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            e[c] = rr + 2 * c + 1 < rank ? e[c] : rr + 2 * c < rank ? e[c] & 0xFFFFu : 0u;
                    }
                }
            }
#pragma unroll
            for (int u = kParts - 1; u >= 0; --u) {
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    if (m == 1 && !two) break;
                    const uint4 lo = *reinterpret_cast<const uint4*>(hs + (size_t)(u * kLoTile + 16 * m + g) * rs + r + 8 * q);
                    const uint4 hi = *reinterpret_cast<const uint4*>(hs + (size_t)(u * kLoTile + 16 * m + g + 8) * rs + r + 8 * q);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        mma_bf16(acc[m][j], lo.x, hi.x, lo.y, hi.y, w[j].x, w[j].y);
                        mma_bf16(acc[m][j], lo.z, hi.z, lo.w, hi.w, w[j].z, w[j].w);
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!cin || g + 8 * i >= s.count) continue;
            float o[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                o[2 * j] = acc[i >> 1][j][(i & 1) * 2];
                o[2 * j + 1] = acc[i >> 1][j][(i & 1) * 2 + 1];
            }
            char* dst = static_cast<char*>(a.out) + ((size_t)s.token[g + 8 * i] * a.N + col) * (kO16 ? 2 : 4);
            if constexpr (kO16) {
                const uint32_t bw[4] = {bv[i][0].x, bv[i][0].y, bv[i][0].z, bv[i][0].w};
                uint32_t w[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const __nv_bfloat162 v = __floats2bfloat162_rn(o[2 * c] + __uint_as_float(bw[c] << 16),
                                                                   o[2 * c + 1] + __uint_as_float(bw[c] & 0xFFFF0000u));
                    w[c] = *reinterpret_cast<const uint32_t*>(&v);
                }
                *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
                const uint32_t bw[8] = {bv[i][0].x, bv[i][0].y, bv[i][0].z, bv[i][0].w,
                                        bv[i][1].x, bv[i][1].y, bv[i][1].z, bv[i][1].w};
                float r[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) r[c] = o[c] + __uint_as_float(bw[c]);
                reinterpret_cast<float4*>(dst)[0] = make_float4(r[0], r[1], r[2], r[3]);
                reinterpret_cast<float4*>(dst)[1] = make_float4(r[4], r[5], r[6], r[7]);
            }
        }
    }
}

}  // namespace coli
