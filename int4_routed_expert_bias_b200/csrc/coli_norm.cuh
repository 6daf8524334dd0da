// coli_norm.cuh -- the residual path around a block (coli_residual_norm):
//   d  = block output; with post_w: d * rsqrt(mean d^2 + eps) * post_w; times the gate
//   r' = residual_scale * r + block_scale * d
//   y  = r' * rsqrt(mean r'^2 + eps) * pre_w
// One pass: a row is read once into registers, both means are reduced over the
// threads that hold it, and r' and y are written from the same registers.  All
// arithmetic is fp32 (y is taken from r' before r' is rounded to the stream's
// type); each output is rounded once.
#pragma once

#include "coli_common.cuh"

namespace coli {

enum { kGateNone = 0, kGateChannel = 1, kGateToken = 2, kGateElement = 3 };

struct NormArgs {
    int T, H;
    int rows;             // rows per block (warp form)
    float eps, inv_h, residual_scale, block_scale;
    int gate, gate_sigmoid;
    const float* post_w;  // [H] or null
    const float* pre_w;   // [H] or null
    const void* d;        // [T, H] block output, or null
    const void* r;        // [T, H] residual
    const void* g;        // gate: [H], [T] or [T, H], type of d
    void* r_out;          // [T, H] or null
    void* y;              // [T, H] or null (with pre_w)
};

// kVec (8 or 1) consecutive values at element i, widened to fp32.
template <bool kBf16, int kVec>
__device__ __forceinline__ void load_vec(const void* p, size_t i, float (&v)[kVec])
{
    if constexpr (kVec == 1) {
        v[0] = kBf16 ? bf16_bits_to_float(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
    } else if constexpr (kBf16) {
        const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(w[j] << 16);
            v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    } else {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        const float4 a = q[0], b = q[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
}

template <bool kBf16, int kVec>
__device__ __forceinline__ void store_vec(void* p, size_t i, const float (&v)[kVec])
{
    if constexpr (kVec == 1) {
        if constexpr (kBf16) static_cast<uint16_t*>(p)[i] = float_to_bf16_bits(v[0]);
        else static_cast<float*>(p)[i] = v[0];
    } else if constexpr (kBf16) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}

// Sum over the threads of a row: a warp, or the block (one barrier; `red` is not reused).
template <bool kWarpRow>
__device__ __forceinline__ float row_sum(float v, float* red)
{
    v = warp_sum(v);
    if constexpr (!kWarpRow) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = blockDim.x >> 5;
        if (lane == 0) red[warp] = v;
        __syncthreads();
        v = warp_sum(lane < n ? red[lane] : 0.f);
    }
    return v;
}

// One row held in d and r (kN vectors of kVec values per thread, `width` threads side by side).
template <bool kD, bool kR, int kVec, int kN, bool kWarpRow>
__device__ __forceinline__ void norm_row(const NormArgs& a, int t, int lane, int width, float (&d)[kN][kVec],
                                         float (&r)[kN][kVec], float (*red)[32])
{
    const size_t row = (size_t)t * a.H;
    float f = a.block_scale;
    if (a.gate == kGateToken) {
        float g[1];
        load_vec<kD, 1>(a.g, t, g);
        f *= a.gate_sigmoid ? 1.0f / (1.0f + expf(-g[0])) : g[0];
    }
    if (a.post_w) {
        float s = 0.f;
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int j = 0; j < kVec; ++j) s = fmaf(d[n][j], d[n][j], s);
        f *= rsqrtf(row_sum<kWarpRow>(s, red[0]) * a.inv_h + a.eps);
    }
    float s = 0.f;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
        const int i = (lane + n * width) * kVec;
        if (i >= a.H) continue;
        float w[kVec];
        if (a.post_w) {
            load_vec<false, kVec>(a.post_w, i, w);
#pragma unroll
            for (int j = 0; j < kVec; ++j) d[n][j] *= w[j];
        }
        if (a.gate == kGateChannel || a.gate == kGateElement) {
            load_vec<kD, kVec>(a.g, a.gate == kGateElement ? row + i : i, w);
#pragma unroll
            for (int j = 0; j < kVec; ++j) d[n][j] *= a.gate_sigmoid ? 1.0f / (1.0f + expf(-w[j])) : w[j];
        }
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            r[n][j] = fmaf(f, d[n][j], a.residual_scale * r[n][j]);
            s = fmaf(r[n][j], r[n][j], s);
        }
        if (a.r_out) store_vec<kR, kVec>(a.r_out, row + i, r[n]);
    }
    if (!a.y) return;
    const float q = rsqrtf(row_sum<kWarpRow>(s, red[1]) * a.inv_h + a.eps);
#pragma unroll
    for (int n = 0; n < kN; ++n) {
        const int i = (lane + n * width) * kVec;
        if (i >= a.H) continue;
        float w[kVec], o[kVec];
        load_vec<false, kVec>(a.pre_w, i, w);
#pragma unroll
        for (int j = 0; j < kVec; ++j) o[j] = r[n][j] * q * w[j];
        store_vec<kD, kVec>(a.y, row + i, o);
    }
}

// kD, kR: bf16 block output / residual.  A block (or, kWarpRow, a warp) per row.
template <bool kD, bool kR, int kVec, int kN, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 256 : 1024) residual_norm_kernel(const __grid_constant__ NormArgs a)
{
    __shared__ float red[2][32];
    const int lane = kWarpRow ? threadIdx.x & 31 : threadIdx.x, width = kWarpRow ? 32 : blockDim.x;
    const int t = kWarpRow ? blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    griddep_wait();
    if (t >= a.T) return;  // whole warps (or none) leave
    float d[kN][kVec], r[kN][kVec];
#pragma unroll
    for (int n = 0; n < kN; ++n) {
        const int i = (lane + n * width) * kVec;
#pragma unroll
        for (int j = 0; j < kVec; ++j) d[n][j] = r[n][j] = 0.f;
        if (i < a.H) {
            if (a.d) load_vec<kD, kVec>(a.d, (size_t)t * a.H + i, d[n]);
            load_vec<kR, kVec>(a.r, (size_t)t * a.H + i, r[n]);
        }
    }
    norm_row<kD, kR, kVec, kN, kWarpRow>(a, t, lane, width, d, r, red);
}

// Long bf16 batches: blocks walk the rows, the next row's loads under way while the
// mean of the current one is reduced.
template <int kN>
__global__ void __launch_bounds__(512) residual_norm_rows_kernel(const __grid_constant__ NormArgs a)
{
    __shared__ float red[2][2][32];
    griddep_wait();
    uint4 pd[kN], pr[kN];  // the next row as it is stored
    auto widen = [](const uint4& u, float (&v)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(w[j] << 16);
            v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    };
    auto load = [&](int t) {
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            const int i = (threadIdx.x + n * blockDim.x) * 8;
            pd[n] = pr[n] = make_uint4(0u, 0u, 0u, 0u);
            if (i < a.H) {
                if (a.d) pd[n] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.d) + (size_t)t * a.H + i);
                pr[n] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.r) + (size_t)t * a.H + i);
            }
        }
    };
    int t = blockIdx.x;
    if (t < a.T) load(t);
    for (int b = 0; t < a.T; t += gridDim.x, b ^= 1) {
        float d[kN][8], r[kN][8];
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            widen(pd[n], d[n]);
            widen(pr[n], r[n]);
        }
        if (t + gridDim.x < a.T) load(t + gridDim.x);
        norm_row<true, true, 8, kN, false>(a, t, threadIdx.x, blockDim.x, d, r, red[b]);
    }
}

}  // namespace coli
