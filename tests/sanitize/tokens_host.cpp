// The token operators' host code (tokens.cpp, adapters.cpp) without a GPU: the launchers
// are stubs that write down, as JSON, what they were asked to launch.  Addresses are never
// dereferenced.
#include <cstdarg>
#include <cstdio>
#include <string>

#include "../../expert_cache_ffn_amd/csrc/tokens_internal.h"

namespace ecf {
namespace {

thread_local std::string t_log, t_error;

std::string num(const char *key, long long v) { return std::string(", \"") + key + "\": " + std::to_string(v); }
std::string at(const char *key, const void *p) { return num(key, (long long)(uintptr_t)p); }
int add(const char *kind, const std::string &s)
{
    t_log += (t_log.empty() ? "{\"kind\": \"" : ", {\"kind\": \"") + std::string(kind) + "\"" + s + "}";
    return ECF_OK;
}

std::string order(const AdapterOrder &o)
{
    return num("t", o.T) + num("n", o.n) + num("wide", o.wide) + at("idx", o.idx) + at("order", o.order) + at("offsets", o.offsets) +
           at("tiles", o.tiles);
}
std::string shrink(const ShrinkCall &c)
{
    return order(c.o) + num("k", c.K) + num("r", c.r) + num("of_b", c.of_b) + num("splits", c.splits) + num("split_k", c.split_k) +
           at("part", c.part);
}
std::string expand(const ExpandCall &c)
{
    return order(c.o) + num("n_out", c.N) + num("r", c.r) + num("of_a", c.of_a) + num("splits", c.splits) + at("part", c.part) +
           at("h", c.h) + at("out", c.out) + num("scaled", c.scaled);
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

int launch_norm_forward(const NormCall &c, hipStream_t) { return add("norm", num("t", c.T) + num("d", c.d) + at("y", c.y)); }
int launch_norm_backward(const NormCall &c, hipStream_t)
{
    return add("norm_backward", num("t", c.T) + num("d", c.d) + at("partial", c.partial) + at("dweight", c.dweight) +
                                    num("parts", norm_partial_rows(c.T, c.d)));
}
int launch_token_sort(const SortCall &c, hipStream_t)
{
    const int s = sort_segments((int64_t)c.T * c.k);
    return add("sort", num("t", c.T) + num("k", c.k) + num("e", c.E) + at("counts", c.counts) + at("offsets", c.offsets) +
                           at("tiles", c.tiles) + at("order", c.order) + at("place", c.place) + at("segments", c.segments) +
                           num("n_segments", s) + num("itself", sort_counts_itself(s)));
}
int launch_dispatch(const MoveCall &c, hipStream_t) { return add("dispatch", num("t", c.T) + num("k", c.k) + num("d", c.d)); }
int launch_combine_tokens(const MoveCall &c, hipStream_t) { return add("combine", num("t", c.T) + num("k", c.k) + num("d", c.d)); }
int launch_combine_backward(const MoveCall &c, hipStream_t)
{
    return add("combine_backward", num("t", c.T) + num("k", c.k) + num("d", c.d));
}
int launch_shrink(const ShrinkCall &c, hipStream_t) { return add("shrink", shrink(c)); }
int launch_expand(const ExpandCall &c, hipStream_t) { return add("expand", expand(c)); }
int launch_few(const ShrinkCall &c, const ExpandCall &x, hipStream_t)
{
    return add("few", num("t", c.o.T) + num("k", c.K) + num("r", c.r) + num("n_out", x.N));
}
int launch_few_shrink(const ShrinkCall &c, hipStream_t) { return add("few_shrink", shrink(c)); }
int launch_few_expand(const ExpandCall &c, hipStream_t) { return add("few_expand", expand(c)); }
int launch_outer(const OuterCall *calls, int n, int chunks, hipStream_t)
{
    for (int i = 0; i < n; ++i) {
        const OuterCall &c = calls[i];
        add("outer", order(c.o) + num("w", c.W) + num("r", c.r) + num("of_b", c.of_b) + num("chunks", chunks) + num("calls", n) +
                         at("g", c.g) + at("slots", c.slots) + at("d", c.d));
    }
    return ECF_OK;
}

}  // namespace ecf

extern "C" {
// What the calls since the last one would have launched: a JSON list.
const char *token_host_launches()
{
    static thread_local std::string out;
    out = "[" + ecf::t_log + "]";
    ecf::t_log.clear();
    return out.c_str();
}
void token_host_grid(long long blocks, unsigned *x, unsigned *y)
{
    const ecf::BlockGrid g = ecf::block_grid(blocks);
    *x = g.x, *y = g.y;
}
const char *token_host_error() { return ecf::t_error.c_str(); }
}
