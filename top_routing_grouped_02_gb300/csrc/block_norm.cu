// The norms around a block (block_norm.cuh): the calls' operands and launch shapes.
#include <algorithm>

#include "block_norm.cuh"

namespace moe {
namespace bn {

bool shape_of(Args &a, int cols, int per_thread, int max_threads, int sms, size_t fixed, size_t stage,
              size_t least, int *groups) {
    // as many groups as have a stage each, rather than fewer with two: they overlap as well
    // (4096 x 4096 fp32 with a full gate, one group of 14 KB rows against two: forward 79 / 58 us)
    Ring r;
    if (!ring_shape({a.T, cols, per_thread, max_threads, kMaxGroups, kRingStages, sms, fixed, 0, stage,
                     std::max(least, stage)}, &r))
        return false;
    a.wpr = r.wpr;
    a.stages = r.stages;
    a.group_bytes = (uint32_t)std::max(least, r.stages * stage);
    *groups = r.groups;
    return true;
}

RowShape row_shape(Args &a, int per_thread) {
    a.wpr = (a.d + per_thread * 32 - 1) / (per_thread * 32);
    RowShape r;
    r.groups = std::max(1, std::min(kRowThreads / (32 * a.wpr), 15));
    // few rows spread over the SMs
    r.groups = (int)std::min<int64_t>(r.groups, std::max<int64_t>(1, (a.T + sm_count() - 1) / sm_count()));
    r.grid = (int)std::min<int64_t>((a.T + r.groups - 1) / r.groups, 4 * sm_count());
    return r;
}

}  // namespace bn

using namespace bn;

int block_norm_partials(int64_t T) {
    return (int)std::min<int64_t>((T + kPhases - 1) / kPhases * kPhases, kLnPartials);
}

cudaError_t launch_block_norm_forward(const BlockNormCall &c, int64_t withheld, cudaStream_t s) {
    Args a{};
    Places places;
    const int es = c.type == MOE_DTYPE_F32 ? 4 : 2;
    auto in = [&](const Matrix &m) {
        places.add(m.p, m.ld, c.d, es, c.T);
        return m.p;
    };
    a.x = in(c.x);
    a.ldx = c.x.ld;
    a.b = in(c.b);
    a.ldb = c.b.ld;
    a.full = c.gate.p != nullptr && c.gate_rows;
    a.gate = a.full ? in(c.gate) : c.gate.p;
    a.ldg = c.gate.ld;
    a.y = const_cast<void *>(in(c.y));
    a.ldy = c.y.ld;
    a.u = const_cast<void *>(in(c.u));
    a.ldu = c.u.ld;
    a.post = c.post;
    a.pre = c.pre;
    a.r_post = c.r_post;
    a.r_pre = c.r_pre;
    a.T = c.T;
    a.d = c.d;
    a.w32 = c.w32;
    a.post_norm = c.post_norm;
    a.pre_norm = c.pre_norm;
    a.scale = c.scale;
    a.eps = c.eps;
    a.withheld = withheld;
    switch (c.type) {
        case MOE_DTYPE_BF16: return forward_type<__nv_bfloat16>(a, places.shift(), s);
        case MOE_DTYPE_F16: return forward_type<__half>(a, places.shift(), s);
        default: return forward_type<float>(a, places.shift(), s);
    }
}

cudaError_t launch_block_norm_backward(const BlockNormCall &c, int64_t withheld, cudaStream_t s) {
    Args a{};
    Places places;
    const int es = c.type == MOE_DTYPE_F32 ? 4 : 2;
    auto in = [&](const Matrix &m) {
        places.add(m.p, m.ld, c.d, es, c.T);
        return m.p;
    };
    auto out = [&](const Matrix &m) { return const_cast<void *>(in(m)); };
    a.x = in(c.x);
    a.ldx = c.x.ld;
    a.b = in(c.b);
    a.ldb = c.b.ld;
    a.full = c.gate.p != nullptr && c.gate_rows;
    a.gate = a.full ? in(c.gate) : c.gate.p;
    a.ldg = c.gate.ld;
    a.dy = in(c.dy);
    a.lddy = c.dy.ld;
    a.du = in(c.du);
    a.lddu = c.du.ld;
    a.dx = out(c.dx);
    a.lddx = c.dx.ld;
    a.db = out(c.db);
    a.lddb = c.db.ld;
    a.dgate = a.full ? out(c.dgate) : const_cast<void *>(c.dgate.p);
    a.lddg = c.dgate.ld;
    a.post = c.post;
    a.pre = c.pre;
    a.r_post = c.r_post;
    a.r_pre = c.r_pre;
    a.T = c.T;
    a.d = c.d;
    a.w32 = c.w32;
    a.post_norm = c.post_norm;
    a.pre_norm = c.pre_norm;
    a.scale = c.scale;
    a.withheld = withheld;
    a.part = c.dpost != nullptr || c.dpre != nullptr ? c.part : nullptr;
    int P = 0;
    const cudaError_t e = c.type == MOE_DTYPE_BF16  ? backward_type<__nv_bfloat16>(a, places.shift(), &P, s)
                          : c.type == MOE_DTYPE_F16 ? backward_type<__half>(a, places.shift(), &P, s)
                                                    : backward_type<float>(a, places.shift(), &P, s);
    if (e != cudaSuccess || a.part == nullptr) return e;
    return launch_weight_reduce(a.part, P, a.d, a.w32 ? MOE_DTYPE_F32 : c.type, c.dpost, c.dpre, s);
}

}  // namespace moe
