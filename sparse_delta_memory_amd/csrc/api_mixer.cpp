// C ABI of the mixer operators (head norms with rotation, slot selection, the gated linear recurrence):
// argument checks on the host, then the kernel launches.
#include <hip/hip_runtime_api.h>

#include <cmath>
#include <cstdint>

#include "sdm.h"
#include "sdm_launch.hpp"

namespace {

using sdm::fail;

// Heads of a norm_rope call: the element path takes a wave per head, and a grid holds fewer than 2^32 work items.
constexpr int64_t kMaxHeads = (int64_t(1) << 26) - 4;   // whole blocks of four waves

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool known(int32_t dtype) { return dtype == SDM_F32 || dtype == SDM_BF16; }
uintptr_t size_of(int32_t dtype) { return dtype == SDM_BF16 ? 2 : 4; }

sdm_status launched(hipError_t e, const char* fn) {
    if (e == hipSuccess) return SDM_OK;
    (void)hipGetLastError();   // reported through the status, not left pending
    return fail(SDM_EHIP, "%s: %s", fn, hipGetErrorString(e));
}

sdm_status set_up(const char* fn, sdm::KernelFamily family) {
    const hipError_t e = sdm::device_setup(nullptr, family);
    if (e != hipSuccess) return fail(SDM_EHIP, "%s: device set-up: %s", fn, hipGetErrorString(e));
    return SDM_OK;
}

sdm_status check_norm_rope(const sdm_norm_rope_io* io, const char* fn) {
    if (io == nullptr) return fail(SDM_EINVAL, "%s: io is NULL", fn);
    if (io->N < 0 || io->Hq < 0 || io->Hk < 0)
        return fail(SDM_ESHAPE, "%s: N = %lld, Hq = %d, Hk = %d", fn, static_cast<long long>(io->N), io->Hq, io->Hk);
    const int64_t heads = static_cast<int64_t>(io->Hq) + io->Hk;
    if (heads < 1 || heads > (1 << 20)) return fail(SDM_ESHAPE, "%s: Hq + Hk = %lld outside 1..2^20", fn, static_cast<long long>(heads));
    if (io->N > kMaxHeads / heads) return fail(SDM_ESHAPE, "%s: N (Hq + Hk) exceeds 2^26 - 4 heads", fn);
    if (io->D < 1 || io->D > 512) return fail(SDM_ESHAPE, "%s: D = %d outside 1..512", fn, io->D);
    if (io->rot < 0 || io->rot > io->D || io->rot % 2 != 0)
        return fail(SDM_ESHAPE, "%s: rot = %d (even, 0..D = %d)", fn, io->rot, io->D);
    if (io->interleaved != 0 && io->interleaved != 1) return fail(SDM_EINVAL, "%s: interleaved = %d (0 or 1)", fn, io->interleaved);
    if (!known(io->dtype) || !known(io->w_dtype)) return fail(SDM_EINVAL, "%s: dtype %d, w_dtype %d", fn, io->dtype, io->w_dtype);
    if (!(io->eps >= 0.0f) || std::isinf(io->eps)) return fail(SDM_EINVAL, "%s: eps = %g (finite, >= 0)", fn, static_cast<double>(io->eps));
    if (io->rot > 0 && io->pos_bytes != 4 && io->pos_bytes != 8)
        return fail(SDM_EINVAL, "%s: pos_bytes = %d (4: int32 positions; 8: int64)", fn, io->pos_bytes);
    if (io->rot > 0 && io->table_rows < 1) return fail(SDM_EINVAL, "%s: table_rows = %lld < 1", fn, static_cast<long long>(io->table_rows));
    if (io->N == 0) return SDM_OK;
    if (io->Hq > 0 && (io->q == nullptr || io->q_out == nullptr)) return fail(SDM_EINVAL, "%s: q and q_out are required", fn);
    if (io->Hk > 0 && (io->k == nullptr || io->k_out == nullptr)) return fail(SDM_EINVAL, "%s: k and k_out are required", fn);
    if (io->rot > 0 && (io->pos == nullptr || io->table == nullptr)) return fail(SDM_EINVAL, "%s: pos and table are required when rot > 0", fn);
    const uintptr_t es = size_of(io->dtype);
    for (const void* p : {io->q, io->k, static_cast<const void*>(io->q_out), static_cast<const void*>(io->k_out)}) {
        if (!aligned(p, es)) return fail(SDM_EALIGN, "%s: a head pointer is not element-aligned", fn);
    }
    if ((io->Hq > 0 && !aligned(io->wq, size_of(io->w_dtype))) || (io->Hk > 0 && !aligned(io->wk, size_of(io->w_dtype))))
        return fail(SDM_EALIGN, "%s: wq or wk is not element-aligned", fn);
    if (io->rot > 0 && (!aligned(io->pos, io->pos_bytes) || !aligned(io->table, 4)))
        return fail(SDM_EALIGN, "%s: pos or table is misaligned", fn);
    return SDM_OK;
}

sdm_status check_slots(const sdm_slot_topk_io* io, const char* fn) {
    if (io == nullptr) return fail(SDM_EINVAL, "%s: io is NULL", fn);
    if (io->N < 0) return fail(SDM_ESHAPE, "%s: N = %lld < 0", fn, static_cast<long long>(io->N));
    if (io->n1 < 1 || io->n1 > 4096 || io->n2 < 1 || io->n2 > 4096)
        return fail(SDM_ESHAPE, "%s: n1 = %d, n2 = %d outside 1..4096", fn, io->n1, io->n2);
    if (io->K < 1 || io->K > 64 || io->K > static_cast<int64_t>(io->n1) * io->n2)
        return fail(SDM_ESHAPE, "%s: K = %d outside 1..min(64, n1 n2)", fn, io->K);
    if (io->N > (int64_t(1) << 40)) return fail(SDM_ESHAPE, "%s: N = %lld > 2^40", fn, static_cast<long long>(io->N));
    if (!known(io->dtype)) return fail(SDM_EINVAL, "%s: dtype %d", fn, io->dtype);
    if (io->idx_bytes != 4 && io->idx_bytes != 8) return fail(SDM_EINVAL, "%s: idx_bytes = %d (4: int32 ids; 8: int64)", fn, io->idx_bytes);
    if (!(io->scale > 0.0f) || std::isinf(io->scale)) return fail(SDM_EINVAL, "%s: scale = %g (finite, > 0)", fn, static_cast<double>(io->scale));
    if (io->chunk_rows < 0 || (io->chunk_rows > 0 && (io->P < 1 || io->stream_offset < 0 || io->stream_offset > (int64_t(1) << 40))))
        return fail(SDM_EINVAL, "%s: chunk_rows = %lld, P = %d, stream_offset = %lld", fn, static_cast<long long>(io->chunk_rows), io->P,
                    static_cast<long long>(io->stream_offset));
    // The last stream's largest id, by division: the product of the largest P and offset passes 64 bits.
    const int64_t slots = static_cast<int64_t>(io->n1) * io->n2, top = io->idx_bytes == 4 ? INT32_MAX : INT64_MAX;
    if (io->chunk_rows > 0 && io->stream_offset > 0 && io->P - 1 > (top - (slots - 1)) / io->stream_offset)
        return fail(SDM_EINVAL, "%s: ids of %d streams of %lld do not fit int%d", fn, io->P, static_cast<long long>(io->stream_offset),
                    8 * io->idx_bytes);
    if (io->N == 0) return SDM_OK;
    if (io->a == nullptr || io->b == nullptr || io->idx == nullptr) return fail(SDM_EINVAL, "%s: a, b and idx are required", fn);
    if (!aligned(io->a, size_of(io->dtype)) || !aligned(io->b, size_of(io->dtype)) || !aligned(io->idx, io->idx_bytes))
        return fail(SDM_EALIGN, "%s: a, b or idx is not element-aligned", fn);
    return SDM_OK;
}

// Alignment of states: 16 bytes where that holds for every row of a pool, else an element's (the rows of odd widths are
// read and written element by element).
uintptr_t state_align(int32_t dk, int32_t dv) { return static_cast<int64_t>(dk) * dv % 4 == 0 ? 16 : 4; }

sdm_status check_heads(int32_t H, int32_t Hk, int32_t dk, int32_t dv, int32_t dtype, float scale, const char* fn) {
    if (H < 1 || Hk < 1 || H % Hk != 0) return fail(SDM_ESHAPE, "%s: H = %d must be a multiple of Hk = %d (both >= 1)", fn, H, Hk);
    if (dk < 1 || dk > 128 || dv < 1 || dv > 128) return fail(SDM_ESHAPE, "%s: dk = %d, dv = %d outside 1..128", fn, dk, dv);
    if (!known(dtype)) return fail(SDM_EINVAL, "%s: dtype %d", fn, dtype);
    if (!std::isfinite(scale)) return fail(SDM_EINVAL, "%s: scale is not finite", fn);
    return SDM_OK;
}

sdm_status check_glr(const sdm_glr_io* io, bool backward, const char* fn) {
    if (io == nullptr) return fail(SDM_EINVAL, "%s: io is NULL", fn);
    if (io->B < 0 || io->T < 0 || io->T > (1 << 30)) return fail(SDM_ESHAPE, "%s: B = %d, T = %d (at most 2^30)", fn, io->B, io->T);
    const sdm_status rc = check_heads(io->H, io->Hk, io->dk, io->dv, io->dtype, io->scale, fn);
    if (rc != SDM_OK) return rc;
    const int64_t bh = static_cast<int64_t>(io->B) * io->H;
    if (bh > (1 << 20) || (io->T > 0 && bh > INT32_MAX / io->T))
        return fail(SDM_ESHAPE, "%s: B H = %lld (at most 2^20), B T H at most 2^31 - 1", fn, static_cast<long long>(bh));
    if (io->B == 0) return SDM_OK;
    if (io->T > 0 && (io->q == nullptr || io->k == nullptr || io->v == nullptr || io->g == nullptr))
        return fail(SDM_EINVAL, "%s: q, k, v and g are required", fn);
    const uintptr_t es = size_of(io->dtype);
    for (const void* p : {io->q, io->k, io->v}) {
        if (!aligned(p, es)) return fail(SDM_EALIGN, "%s: q, k or v is not element-aligned", fn);
    }
    if (!aligned(io->g, 4) || !aligned(io->lens, 4)) return fail(SDM_EALIGN, "%s: g or lens is misaligned", fn);
    const uintptr_t sa = state_align(io->dk, io->dv);
    if (!aligned(io->state, sa)) return fail(SDM_EALIGN, "%s: state must be %d-byte aligned", fn, static_cast<int>(sa));
    const size_t need = sdm::glr_workspace_bytes(io, backward);
    if (need > 0 && (io->workspace == nullptr || io->workspace_bytes < need))
        return fail(SDM_EWORKSPACE, "%s: workspace needs %zu bytes, got %zu", fn, need, io->workspace == nullptr ? size_t(0) : io->workspace_bytes);
    if (!aligned(io->workspace, 256)) return fail(SDM_EALIGN, "%s: workspace must be 256-byte aligned", fn);
    return SDM_OK;
}

}  // namespace

extern "C" {

sdm_status sdm_norm_rope(const sdm_norm_rope_io* io, hipStream_t st) {
    sdm::clear_error();
    const sdm_status rc = check_norm_rope(io, "sdm_norm_rope");
    if (rc != SDM_OK || io->N == 0) return rc;
    return launched(sdm::norm_rope_launch(io, st), "sdm_norm_rope");
}

size_t sdm_norm_rope_workspace(const sdm_norm_rope_io* io) {
    if (io == nullptr || io->N < 1 || io->Hq < 0 || io->Hk < 0 || io->D < 1 || io->D > 512) return 0;
    const int64_t heads = static_cast<int64_t>(io->Hq) + io->Hk;
    if (heads < 1 || heads > (1 << 20) || io->N > kMaxHeads / heads) return 0;
    return sdm::norm_rope_back_workspace(io->N, static_cast<int>(heads), io->D);
}

sdm_status sdm_norm_rope_backward(const sdm_norm_rope_io* io, const sdm_norm_rope_grad* g, hipStream_t st) {
    sdm::clear_error();
    const char* fn = "sdm_norm_rope_backward";
    const sdm_status rc = check_norm_rope(io, fn);
    if (rc != SDM_OK) return rc;
    if (g == nullptr) return fail(SDM_EINVAL, "%s: grad is NULL", fn);
    if (io->N > 0 && ((io->Hq > 0 && g->dq == nullptr) || (io->Hk > 0 && g->dk == nullptr)))
        return fail(SDM_EINVAL, "%s: dq and dk are required", fn);
    if (!aligned(g->dq, size_of(io->dtype)) || !aligned(g->dk, size_of(io->dtype)) || !aligned(g->dwq, 4) || !aligned(g->dwk, 4))
        return fail(SDM_EALIGN, "%s: a gradient is not element-aligned", fn);
    const size_t need = sdm_norm_rope_workspace(io);
    if (need > 0 && (g->workspace == nullptr || g->workspace_bytes < need))   // no token: the weights' gradients are 0
        return fail(SDM_EWORKSPACE, "%s: workspace needs %zu bytes, got %zu", fn, need, g->workspace == nullptr ? size_t(0) : g->workspace_bytes);
    if (!aligned(g->workspace, 16)) return fail(SDM_EALIGN, "%s: workspace is not 16-byte aligned", fn);
    return launched(sdm::norm_rope_back_launch(io, g, st), fn);
}

sdm_status sdm_slot_topk(const sdm_slot_topk_io* io, hipStream_t st) {
    sdm::clear_error();
    const char* fn = "sdm_slot_topk";
    const sdm_status rc = check_slots(io, fn);
    if (rc != SDM_OK) return rc;
    if (!known(io->val_dtype)) return fail(SDM_EINVAL, "%s: val_dtype %d", fn, io->val_dtype);
    if (io->N == 0) return SDM_OK;
    if (io->val == nullptr) return fail(SDM_EINVAL, "%s: val is required", fn);
    if (!aligned(io->val, size_of(io->val_dtype))) return fail(SDM_EALIGN, "%s: val is not element-aligned", fn);
    return launched(sdm::slot_topk_launch(io, st), fn);
}

sdm_status sdm_slot_topk_backward(const sdm_slot_topk_io* io, const sdm_slot_topk_grad* g, hipStream_t st) {
    sdm::clear_error();
    const char* fn = "sdm_slot_topk_backward";
    sdm_status rc = check_slots(io, fn);
    if (rc != SDM_OK) return rc;
    if (g == nullptr) return fail(SDM_EINVAL, "%s: grad is NULL", fn);
    if (io->N == 0) return SDM_OK;
    if (g->dval == nullptr) return fail(SDM_EINVAL, "%s: dval is required", fn);
    if (!aligned(g->dval, 4) || !aligned(g->da, size_of(io->dtype)) || !aligned(g->db, size_of(io->dtype)))
        return fail(SDM_EALIGN, "%s: dval, da or db is not element-aligned", fn);
    if (g->da == nullptr && g->db == nullptr) return SDM_OK;
    rc = set_up(fn, sdm::KernelFamily::slots);
    if (rc != SDM_OK) return rc;
    return launched(sdm::slot_topk_back_launch(io, g, st), fn);
}

size_t sdm_glr_workspace(const sdm_glr_io* io, int32_t backward) {
    if (io == nullptr || io->B < 1 || io->T < 0 || io->T > (1 << 30) || io->H < 1 || io->Hk < 1 || io->H % io->Hk != 0 || io->dk < 1 || io->dk > 128 ||
        io->dv < 1 || io->dv > 128)
        return 0;
    const int64_t bh = static_cast<int64_t>(io->B) * io->H;
    if (bh > (1 << 20) || (io->T > 0 && bh > INT32_MAX / io->T)) return 0;
    return sdm::glr_workspace_bytes(io, backward != 0);
}

sdm_status sdm_glr_forward(const sdm_glr_io* io, hipStream_t st) {
    sdm::clear_error();
    const char* fn = "sdm_glr_forward";
    sdm_status rc = check_glr(io, false, fn);
    if (rc != SDM_OK || io->B == 0) return rc;
    if (io->T > 0 && io->o == nullptr) return fail(SDM_EINVAL, "%s: o is required", fn);
    if (!aligned(io->o, size_of(io->dtype))) return fail(SDM_EALIGN, "%s: o is not element-aligned", fn);
    const uintptr_t sa = state_align(io->dk, io->dv);
    if (!aligned(io->last, sa)) return fail(SDM_EALIGN, "%s: last must be %d-byte aligned", fn, static_cast<int>(sa));
    if (io->last != nullptr && io->last == io->state) return fail(SDM_EINVAL, "%s: last must not be state", fn);
    rc = set_up(fn, sdm::KernelFamily::recurrence);
    if (rc != SDM_OK) return rc;
    return launched(sdm::glr_forward_launch(io, st), fn);
}

sdm_status sdm_glr_backward(const sdm_glr_io* io, const sdm_glr_grad* g, hipStream_t st) {
    sdm::clear_error();
    const char* fn = "sdm_glr_backward";
    sdm_status rc = check_glr(io, true, fn);
    if (rc != SDM_OK) return rc;
    if (g == nullptr) return fail(SDM_EINVAL, "%s: grad is NULL", fn);
    if (io->B == 0) return SDM_OK;
    if (io->T > 0 && (g->d_o == nullptr || g->dq == nullptr || g->dk == nullptr || g->dv == nullptr || g->dg == nullptr))
        return fail(SDM_EINVAL, "%s: d_o, dq, dk, dv and dg are required", fn);
    const uintptr_t es = size_of(io->dtype);
    if (!aligned(g->d_o, es)) return fail(SDM_EALIGN, "%s: d_o is not element-aligned", fn);
    const uintptr_t sa = state_align(io->dk, io->dv);
    if (!aligned(g->dq, 16) || !aligned(g->dk, 16) || !aligned(g->dv, 16) || !aligned(g->dg, 4) || !aligned(g->d_last, sa) ||
        !aligned(g->d_state, sa))
        return fail(SDM_EALIGN, "%s: dq, dk and dv must be 16-byte aligned, d_last and d_state %d", fn, static_cast<int>(sa));
    if (g->d_state != nullptr && (g->d_state == g->d_last || g->d_state == io->state))
        return fail(SDM_EINVAL, "%s: d_state must not be d_last or state", fn);   // every segment starts from those
    rc = set_up(fn, sdm::KernelFamily::recurrence);
    if (rc != SDM_OK) return rc;
    return launched(sdm::glr_backward_launch(io, g, st), fn);
}

sdm_status sdm_glr_step(const sdm_glr_step_io* io, hipStream_t st) {
    sdm::clear_error();
    const char* fn = "sdm_glr_step";
    if (io == nullptr) return fail(SDM_EINVAL, "%s: io is NULL", fn);
    if (io->B < 0) return fail(SDM_ESHAPE, "%s: B = %d < 0", fn, io->B);
    const sdm_status rc = check_heads(io->H, io->Hk, io->dk, io->dv, io->dtype, io->scale, fn);
    if (rc != SDM_OK) return rc;
    if (static_cast<int64_t>(io->B) * io->H > (1 << 23)) return fail(SDM_ESHAPE, "%s: B H exceeds 2^23", fn);
    if (io->rows < 0 || (io->slots == nullptr && io->rows < io->B))
        return fail(SDM_EINVAL, "%s: %lld state rows for %d requests", fn, static_cast<long long>(io->rows), io->B);
    if (io->B == 0) return SDM_OK;
    if (io->q == nullptr || io->k == nullptr || io->v == nullptr || io->g == nullptr || io->o == nullptr ||
        (io->rows > 0 && (io->state == nullptr || io->new_state == nullptr)))
        return fail(SDM_EINVAL, "%s: q, k, v, g, o, state and new_state are required", fn);
    const uintptr_t es = size_of(io->dtype);
    for (const void* p : {io->q, io->k, io->v, static_cast<const void*>(io->o)}) {
        if (!aligned(p, es)) return fail(SDM_EALIGN, "%s: q, k, v or o is not element-aligned", fn);
    }
    if (!aligned(io->g, 4) || !aligned(io->slots, 4)) return fail(SDM_EALIGN, "%s: g or slots is misaligned", fn);
    const uintptr_t sa = state_align(io->dk, io->dv);
    if (!aligned(io->state, sa) || !aligned(io->new_state, sa))
        return fail(SDM_EALIGN, "%s: state and new_state must be %d-byte aligned", fn, static_cast<int>(sa));
    return launched(sdm::glr_step_launch(io, st), fn);
}

}  // extern "C"
