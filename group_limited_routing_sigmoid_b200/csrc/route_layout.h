// How the experts of a row lie in a warp (route_scores.cu).  Plain C++, so that
// the whole documented range can be walked on the host.
#pragma once

#ifdef __CUDACC__
#define BEAM_HD __host__ __device__ __forceinline__
#else
#define BEAM_HD inline
#endif

namespace beam {

struct RouteLayout {
    int lanes_log;  // log2 of the lanes a group has (5 when no groups are dropped)
    int size;       // experts a group (E when no groups are dropped)
    int epl;        // experts a lane
    int regs;       // the kernel's registers for them, at least epl: 1, 2, 4, 8, 16, 32 or 64
};

// With groups to drop each gets a power of two of lanes, as many as fit.  Where
// n_group is no power of two, lanes are left over and the others own up to 60
// experts (17 groups of 60: one lane each; 9 of 113: two of 57).
BEAM_HD RouteLayout route_layout(int E, int n_group, int topk_group)
{
    RouteLayout l{};
    const bool groups = topk_group < n_group;
    l.lanes_log = 5;
    while (groups && n_group << l.lanes_log > 32) --l.lanes_log;
    l.size = groups ? E / n_group : E;
    l.epl = (l.size + (1 << l.lanes_log) - 1) >> l.lanes_log;
    if (l.epl > 2) l.epl = (l.epl + 3) / 4 * 4;   // whole 16-byte loads
    l.regs = 1;
    while (l.regs < l.epl) l.regs *= 2;
    return l;
}

// A lane's experts: `mine` of them from e0.
struct Span {
    int e0, mine;
    BEAM_HD Span(int lane, int lanes_log, int size, int epl, int E)
    {
        const int sub = (lane & ((1 << lanes_log) - 1)) * epl, left = size - sub;
        e0 = (lane >> lanes_log) * size + sub;
        mine = e0 >= E || left <= 0 ? 0 : left < epl ? left : epl;
    }
};

}  // namespace beam
