// blocknorm.cuh -- what the block norm's forward (k_blocknorm.cu) and backward (k_blocknorm_bwd.cu) share.
#pragma once

#include "internal.h"
#include "launch.cuh"
#include "rows.cuh"

namespace repro {
namespace {

template <int W, int G2> __device__ __forceinline__ void gain_row(const float* g, const RowLane& r, u64 (&v)[G2])
{
    load_row<W, false>(g, r, v);
    flush_row(v);
}

inline bool rows4_or_none(const void* p, int64_t ld, size_t bytes)
{
    return !p || ((reinterpret_cast<uintptr_t>(p) % (4 * bytes)) == 0 && ld % 4 == 0);
}

inline void set_up(NormArgs& a)
{
    const size_t t = a.type == 0 ? 4 : 2, u = a.u_type == 0 ? 4 : 2;
    a.tpr = row_threads(a.D);
    a.inv = (a.D & (a.D - 1)) == 0 ? 1.0f / (float)a.D : 0.0f;
    a.vec = rows4_or_none(a.x, a.x_ld, t) && rows4_or_none(a.y, a.y_ld, t) && rows4_or_none(a.h, a.h_ld, t) &&
            rows4_or_none(a.u, a.u_ld, u) && rows4_or_none(a.dh, a.dh_ld, t) && rows4_or_none(a.du, a.du_ld, u) &&
            rows4_or_none(a.hs, a.hs_ld, t) && rows4_or_none(a.dx, a.dx_ld, t) && rows4_or_none(a.dy, a.dy_ld, t) &&
            (a.gate_rows ? rows4_or_none(a.gate, a.gate_ld, t) && rows4_or_none(a.dgate, a.dgate_ld, t)
                         : rows4_or_none(a.gate, 0, 4)) &&
            rows4_or_none(a.gain_post, 0, 4) && rows4_or_none(a.gain_pre, 0, 4);
}

inline int check_of(const NormArgs& a)
{
    return !a.vec || a.D % 4 != 0 ? ELEMENTS : a.D == (int64_t)16 * row_threads(a.D) ? WHOLE : GROUPS;
}

// threads of a CTA and CTAs of a grid for so many rows or chunks
inline dim3 grid_of(const NormArgs& a, int64_t items, int& threads)
{
    threads = a.tpr < 128 ? 128 : a.tpr;
    const int64_t per = threads / a.tpr, ctas = (items + per - 1) / per, most = (int64_t)num_sms() * 64;
    count_launches(1);
    return dim3((unsigned)(ctas < most ? ctas : most));
}

} // namespace
} // namespace repro
