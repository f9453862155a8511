// The dense operators' host code (dense.cpp, dense_plan.cpp) without a GPU: the
// launchers are stubs that write down, as JSON, what they were asked to launch
// and which kernels the plan gives it.  Addresses are never dereferenced.
#include <cstdarg>
#include <cstdio>
#include <string>

#include "../../expert_cache_ffn_amd/csrc/dense_internal.h"

namespace ecf {
namespace {

thread_local std::string t_log, t_error;
int g_cus = 256;

std::string num(const char *key, long long v) { return std::string("\"") + key + "\": " + std::to_string(v) + ", "; }

std::string operand(const DenseGemm &g)
{
    return num("m", g.M) + num("n", g.N) + num("k", g.K) + num("gated", g.gated) + num("at", g.a_t) + num("bt", g.b_t) +
           num("lda", g.lda) + num("a0", (long long)(uintptr_t)g.a[0]) + num("a1", (long long)(uintptr_t)g.a[1]) +
           num("unscale", (long long)(uintptr_t)g.unscale);
}

// bytes of the partial sums that a split product writes: fp32 [split][half or projection][M][N rounded up to 8]
long long partials(const DenseGemm &g, int splits)
{
    return splits > 1 ? (long long)splits * (g.gated ? 2 : g.mhalves) * g.M * ((g.N + 7) / 8 * 8) * 4 : 0;
}

void add(const std::string &s)
{
    t_log += (t_log.empty() ? "{" : ", {") + s.substr(0, s.size() - 2) + "}";
}

}  // namespace

int set_error(int code, const char *fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    t_error = buf;
    return code;
}

int launch_dense_gemm(const DenseGemm &g, void *ws, size_t room, hipStream_t)
{
    const DenseChoice c = choose_gemm(g, g_cus, room);
    std::string s = operand(g) + num("ws", (long long)(uintptr_t)ws) + num("room", (long long)room);
    if (c.kind == DenseChoice::kFew)
        s += "\"kind\": \"few\", " + num("rows", c.few.rows) + num("groups", c.few.groups) + num("waves", c.few.waves);
    else if (c.kind == DenseChoice::kShort)
        s += "\"kind\": \"short\", ";
    else
        s += "\"kind\": \"tiles\", " + num("tile", c.tiles.tile) + num("splits", c.tiles.splits) + num("dma", c.tiles.dma) +
             num("partials", partials(g, c.tiles.splits));
    add(s);
    return ECF_OK;
}

int launch_dense_backward(const DenseGemm *gx, const DenseGemm *gw, const DenseColsum &, void *ws, size_t room,
                          hipStream_t st)
{
    DensePair p;
    if (gx && gw && choose_pair(*gx, *gw, g_cus, room, &p)) {
        add(operand(*gx) + num("ws", (long long)(uintptr_t)ws) + num("room", (long long)room) + num("at_w", (long long)p.at_w) +
            "\"kind\": \"pair\", " + num("tile", p.x.tile) +
            num("dma", p.x.dma) + num("splits", p.x.splits) + num("splits_w", p.splits_w) +
            num("partials", partials(*gx, p.x.splits)) + num("partials_w", partials(*gw, p.splits_w)));
        return ECF_OK;
    }
    if (gx)
        launch_dense_gemm(*gx, ws, room, st);
    return gw ? launch_dense_gemm(*gw, ws, room, st) : ECF_OK;
}

int64_t dense_grad_max_row_blocks(int64_t T) { return (T + 31) / 32; }
int64_t dense_grad_col_blocks(int64_t I) { return (I + 63) / 64; }

int launch_dense_grad(const DenseGrad &g, DenseColsum *, hipStream_t)
{
    add("\"kind\": \"grad\", " + num("dz", (long long)(uintptr_t)g.dz) + num("pitch", g.pitch) +
        num("scaled", g.scaled) + num("dz_w", (long long)(uintptr_t)g.dz_w) +
        num("row_tops", (long long)(uintptr_t)g.row_tops) + num("col_tops", (long long)(uintptr_t)g.col_tops) +
        num("row_inverse", (long long)(uintptr_t)g.row_inverse) + num("col_inverse", (long long)(uintptr_t)g.col_inverse) +
        num("sums", g.want_sums) + num("partial", (long long)(uintptr_t)g.partial));
    return ECF_OK;
}

}  // namespace ecf

extern "C" {
// What the calls since the last one would have launched: a JSON list.
const char *dense_host_launches()
{
    static thread_local std::string out;
    out = "[" + ecf::t_log + "]";
    ecf::t_log.clear();
    return out.c_str();
}
const char *dense_host_error() { return ecf::t_error.c_str(); }
void dense_host_cus(int cus) { ecf::g_cus = cus; }
}
