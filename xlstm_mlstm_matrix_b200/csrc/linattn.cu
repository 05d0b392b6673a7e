// Linear attention with a decay per head: segment plan, workspace and the order of the launches.
#include "linattn.cuh"

namespace xlstm {
namespace {

// Tokens of a segment.
int segment(const LinAttnArgs &a) {
    if (a.dtype != XLSTM_BF16) return 128;
    return (size_t)a.dqk * a.dv > 128 * 128 ? 256 : 512;
}

struct Plan {
    int G, nseg;
    size_t sums, states;     // bytes of the segments' sums (fp32) and of their entering states, one direction
};
Plan plan(const LinAttnArgs &a) {
    Plan p;
    p.G = segment(a);
    p.nseg = (a.T + p.G - 1) / p.G;
    const size_t n = (size_t)a.B * a.H * p.nseg * a.dv * a.dqk;
    p.sums = 4 * n;
    p.states = a.dtype == XLSTM_BF16 ? 2 * n : 0;     // fp32 states take the sums' place
    return p;
}

// The entering states of all segments (and the chain's end) in one direction; returns where they are.
cudaError_t states(const LinAttnArgs &a, const Plan &pl, bool rev, char *ws, const void *&where, cudaStream_t s) {
    const bool bf16 = a.dtype == XLSTM_BF16;
    LinStateP p{};
    p.B = a.B; p.H = a.H; p.T = a.T; p.dqk = a.dqk; p.dv = a.dv; p.G = pl.G; p.nseg = pl.nseg;
    p.rev = rev; p.scale = a.scale; p.log_decay = a.log_decay; p.lens = a.lens;
    p.z = rev ? a.do_ : a.v;
    p.y = rev ? a.q : a.k;
    p.init = rev ? a.dC1 : a.C0;
    p.last = rev ? a.dC0 : a.C1;
    p.sums = reinterpret_cast<float *>(ws);
    p.states = bf16 ? ws + pl.sums : ws;
    where = p.states;
    if (p.nseg == 1 && !p.init && !p.last) return cudaSuccess;   // nothing enters, nothing is handed on
    if (p.nseg > 1 || p.last) {
        const cudaError_t e = bf16 ? linattn_sums_tc(p, a.status, s) : linattn_sums_simt(p, s);
        if (e != cudaSuccess) return e;
    }
    return linattn_chain(p, bf16, s);
}

// out_t = scale sum l^{|t-s|} (x_t.y_s) z_s + rho_t (entering state) x_t
cudaError_t tile(const LinAttnArgs &a, const Plan &pl, bool rev, const void *x, const void *y, const void *z, int dx,
                 int dz, bool state_t, const void *states, void *out, cudaStream_t s) {
    LinTileP p{};
    p.B = a.B; p.H = a.H; p.T = a.T; p.dx = dx; p.dz = dz; p.G = pl.G; p.nseg = pl.nseg;
    p.rev = rev; p.state_t = state_t; p.has_init = rev ? a.dC1 != nullptr : a.C0 != nullptr;
    p.scale = a.scale; p.x = x; p.y = y; p.z = z; p.log_decay = a.log_decay; p.lens = a.lens;
    p.states = states; p.out = out;
    return a.dtype == XLSTM_BF16 ? linattn_tile_tc(p, a.status, s) : linattn_tile_simt(p, s);
}

}  // namespace

size_t linattn_workspace_bytes(const LinAttnArgs &a, bool backward) {
    const Plan p = plan(a);
    return (backward ? 2 : 1) * (p.sums + p.states);
}

cudaError_t launch_linattn_fwd(const LinAttnArgs &a, cudaStream_t s) {
    const Plan pl = plan(a);
    const void *C;
    const cudaError_t e = states(a, pl, false, static_cast<char *>(a.workspace), C, s);
    return e != cudaSuccess ? e : tile(a, pl, false, a.q, a.k, a.v, a.dqk, a.dv, false, C, a.o, s);
}

cudaError_t launch_linattn_bwd(const LinAttnArgs &a, cudaStream_t s) {
    const Plan pl = plan(a);
    char *ws = static_cast<char *>(a.workspace);
    const void *C, *E;
    cudaError_t e = states(a, pl, false, ws, C, s);
    if (e == cudaSuccess) e = states(a, pl, true, ws + pl.sums + pl.states, E, s);
    if (e == cudaSuccess) e = tile(a, pl, false, a.do_, a.v, a.k, a.dv, a.dqk, true, C, a.dq, s);
    if (e == cudaSuccess) e = tile(a, pl, true, a.v, a.do_, a.q, a.dv, a.dqk, true, E, a.dk, s);
    if (e == cudaSuccess) e = tile(a, pl, true, a.k, a.q, a.do_, a.dqk, a.dv, false, E, a.dv_, s);
    return e;
}

}  // namespace xlstm
