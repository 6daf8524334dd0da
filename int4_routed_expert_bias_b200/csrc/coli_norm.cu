// coli_norm.cu -- host side of the residual path around a block (coli_residual_norm).
#include <algorithm>
#include <cmath>

#include "coli_host.h"
#include "coli_norm.cuh"

using namespace coli;

namespace {

constexpr int kSms = 148;                    // grid sizing (B200)
constexpr size_t kWalkFrom = (size_t)8 << 20;  // values of a batch from which blocks walk its rows
constexpr int kMaxWalkVecs = 1024;

template <bool kD, bool kR>
cudaError_t launch(const NormArgs& a, cudaStream_t s)
{
    // Rows that are whole 16-byte vectors in every type (the pointers are 16-byte aligned) are read so;
    // other widths value by value.
    auto go = [&](auto kern, int blocks, int threads) { return launch_pdl(kern, dim3(blocks), threads, 0, s, a); };
    const int eighth = (a.T + 7) / 8;  // warp form: eight rows per block
    if (a.H % 8 == 0) {
        const int nv = a.H / 8;
        if (nv <= 32) return go(residual_norm_kernel<kD, kR, 8, 1, true>, eighth, 256);
        if (nv <= 64) return go(residual_norm_kernel<kD, kR, 8, 2, true>, eighth, 256);
        const int threads = ((nv + 1) / 2 + 31) / 32 * 32;
        // Blocks that walk the rows with the next row's loads under way win for bf16 where the traffic does not stay in
        // L2 and only one mean is reduced (4800 x 6144: 37.9 us, a block per row 44.7; 9600 x 2048: 25.7, 28.1).  With
        // the norm of the block's output too, more blocks per SM hide its second reduction better (4800 x 8192: 76 us
        // against 95), and fp32 rows keep enough bytes under way without (9600 x 6144, fp32 residual: 103 against 128).
        if constexpr (kD && kR)
            if (!a.post_w && nv <= kMaxWalkVecs && (size_t)a.T * a.H >= kWalkFrom)
                return go(residual_norm_rows_kernel<2>, kSms * std::max(1, 800 / threads), threads);
        return go(residual_norm_kernel<kD, kR, 8, 2, false>, a.T, threads);
    }
    if (a.H <= 128) return go(residual_norm_kernel<kD, kR, 1, 4, true>, eighth, 256);
    if (a.H <= 4096) return go(residual_norm_kernel<kD, kR, 1, 4, false>, a.T, ((a.H + 3) / 4 + 31) / 32 * 32);
    return go(residual_norm_kernel<kD, kR, 1, 16, false>, a.T, 1024);
}

coli_status check_norm(const coli_block_norm* n)
{
    if (!n) return fail(COLI_ERR_INVALID_ARG, "norm is NULL");
    if (n->hidden < 1 || n->hidden > 16384) return fail(COLI_ERR_INVALID_ARG, "hidden=%d outside [1, 16384]", n->hidden);
    if (!(n->eps >= 0.f) || !std::isfinite(n->eps)) return fail(COLI_ERR_INVALID_ARG, "eps is negative or not finite");
    if ((int)n->gate < 0 || (int)n->gate > 3) return fail(COLI_ERR_INVALID_ARG, "unknown gate %d", (int)n->gate);
    if (n->gate_sigmoid != 0 && n->gate_sigmoid != 1)
        return fail(COLI_ERR_INVALID_ARG, "gate_sigmoid=%d (0 or 1)", n->gate_sigmoid);
    if (!std::isfinite(n->residual_scale) || !std::isfinite(n->block_scale))
        return fail(COLI_ERR_INVALID_ARG, "residual_scale / block_scale not finite");
    if (!aligned(n->post_w, 16) || !aligned(n->pre_w, 16))
        return fail(COLI_ERR_INVALID_ARG, "norm.post_w / norm.pre_w not 16-byte aligned");
    return COLI_OK;
}

}  // namespace

coli_status coli::check_residual_norm(const coli_block_norm* n, const void* block_out, coli_dtype xt, const void* residual,
                                      coli_dtype rt, const void* gate, int T, void* residual_out, void* normed_out)
{
    coli_status st = check_norm(n);
    if (st != COLI_OK) return st;
    if (!known_dtype(xt)) return fail(COLI_ERR_INVALID_ARG, "unknown activation dtype %d", (int)xt);
    if (!known_dtype(rt)) return fail(COLI_ERR_INVALID_ARG, "unknown residual dtype %d", (int)rt);
    if (T < 0 || T > kMaxTokens) return fail(COLI_ERR_INVALID_ARG, "T=%d outside [0, %d]", T, kMaxTokens);
    if (T == 0) return COLI_OK;  // (empty tensors have no address)
    if (!block_out && (n->post_w || n->gate != COLI_GATE_NONE))
        return fail(COLI_ERR_INVALID_ARG, "block_out is NULL, but the norm has weights or a gate for it");
    if (!residual_out && !normed_out) return fail(COLI_ERR_INVALID_ARG, "neither residual_out nor normed_out is given");
    if ((normed_out != nullptr) != (n->pre_w != nullptr))
        return fail(COLI_ERR_INVALID_ARG, "normed_out and norm.pre_w go together");
    if (!residual) return fail(COLI_ERR_INVALID_ARG, "residual is NULL");
    if (n->gate != COLI_GATE_NONE && !gate) return fail(COLI_ERR_INVALID_ARG, "gate is NULL");
    const void* ptrs[] = {block_out, residual, residual_out, normed_out, gate};
    for (const void* p : ptrs)
        if (!aligned(p, 16)) return fail(COLI_ERR_INVALID_ARG, "tensor not 16-byte aligned");
    // A thread reads its values of every input before it writes them, so an output may be one of the inputs;
    // anything else in common would be read after it is overwritten.
    const size_t nx = (size_t)T * n->hidden * dtype_size(xt), nr = (size_t)T * n->hidden * dtype_size(rt);
    const size_t ng = n->gate == COLI_GATE_ELEMENT ? nx : (size_t)(n->gate == COLI_GATE_CHANNEL ? n->hidden : T) * dtype_size(xt);
    const bool gate_same = n->gate == COLI_GATE_ELEMENT;
    const struct {
        const void* p;
        size_t bytes;
        coli_dtype t;
        bool may_be_same;
    } in[] = {{block_out, nx, xt, true},
              {residual, nr, rt, true},
              {n->gate == COLI_GATE_NONE ? nullptr : gate, ng, xt, gate_same},
              {n->post_w, (size_t)n->hidden * 4, COLI_F32, false},
              {n->pre_w, (size_t)n->hidden * 4, COLI_F32, false}};
    for (const auto& x : in) {
        if (residual_out && overlap(x.p, x.bytes, residual_out, nr) && !(x.may_be_same && x.p == residual_out && x.t == rt))
            return fail(COLI_ERR_INVALID_ARG, "residual_out overlaps an input without being the same tensor");
        if (normed_out && overlap(x.p, x.bytes, normed_out, nx) && !(x.may_be_same && x.p == normed_out && x.t == xt))
            return fail(COLI_ERR_INVALID_ARG, "normed_out overlaps an input without being the same tensor");
    }
    if (overlap(residual_out, nr, normed_out, nx)) return fail(COLI_ERR_INVALID_ARG, "residual_out and normed_out overlap");
    return COLI_OK;
}

extern "C" coli_status coli_residual_norm(const coli_block_norm* n, const void* block_out, coli_dtype xt,
                                          const void* residual, coli_dtype rt, const void* gate, int T,
                                          void* residual_out, void* normed_out, cudaStream_t stream)
{
    coli_status st = check_residual_norm(n, block_out, xt, residual, rt, gate, T, residual_out, normed_out);
    if (st != COLI_OK || T == 0) return st;
    NormArgs a{};
    a.T = T, a.H = n->hidden;
    a.eps = n->eps, a.inv_h = 1.0f / (float)n->hidden;
    a.residual_scale = n->residual_scale, a.block_scale = n->block_scale;
    a.gate = (int)n->gate, a.gate_sigmoid = n->gate_sigmoid;
    a.post_w = n->post_w, a.pre_w = n->pre_w;
    a.d = block_out, a.r = residual, a.g = gate, a.r_out = residual_out, a.y = normed_out;
    const bool d16 = xt == COLI_BF16, r16 = rt == COLI_BF16;
    const cudaError_t e = d16 ? (r16 ? launch<true, true>(a, stream) : launch<true, false>(a, stream))
                              : (r16 ? launch<false, true>(a, stream) : launch<false, false>(a, stream));
    return e == cudaSuccess ? COLI_OK : cuda_fail(e, "residual norm launch");
}
