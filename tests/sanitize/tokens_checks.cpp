// A sweep of the token operators' entry points under the sanitizers: sizes from one to the
// largest, every type, missing operands and workspaces, on stub launchers.
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "../../include/ecf.h"

extern "C" const char *token_host_launches();

namespace {
char *const base = (char *)((size_t)1 << 40);
void *mem(int i) { return base + (size_t)i * ((size_t)1 << 36); }
}  // namespace

int main()
{
    const int sizes[] = {1, 7, 8, 64, 65, 257, 2048, 2049, 16384, 200001, 1 << 22, 0, -1, (1 << 22) + 1};
    const int tokens[] = {0, 1, 16, 64, 65, 500, 8192, 100001, 1 << 21, 1 << 22, -1};
    const int experts[] = {1, 8, 256, 1024, 0, 1025};
    long done = 0, fine = 0;
    for (int dt : {ECF_F32, ECF_BF16, ECF_F16, ECF_MXFP4})
        for (int d : sizes)
            for (int T : tokens) {
                ecf_norm_args n;
                std::memset(&n, 0, sizeof n);
                n.hidden = d, n.dtype = dt, n.sum_dtype = done % 2 ? ECF_F32 : dt, n.weight_dtype = n.wgrad_dtype = dt;
                n.d_weight = done % 3 ? mem(1) : nullptr;
                n.d_x = mem(2), n.d_residual = mem(3), n.d_sum = mem(4), n.d_y = mem(5), n.d_rstd = (float *)mem(6);
                n.ld_x = done % 5 ? 0 : (int64_t)d + 3;
                fine += ecf_norm_forward(&n, T) == ECF_OK;
                n.d_dy = mem(7), n.d_dsum = mem(8), n.d_dx = mem(9), n.d_ds = mem(10), n.d_dweight = mem(11), n.d_ws = mem(12);
                const size_t ws = ecf_norm_workspace_bytes(d, T, 1);
                n.ws_bytes = ws == SIZE_MAX ? 0 : ws;
                fine += ecf_norm_backward(&n, T) == ECF_OK;
                for (int E : experts)
                    for (int k : {1, 6, 32, 33}) {
                        ecf_sort_args s;
                        std::memset(&s, 0, sizeof s);
                        s.n_experts = E, s.top_k = k, s.idx_bytes = done % 2 ? 4 : 8, s.d_idx = mem(1);
                        s.d_counts = (int32_t *)mem(2), s.d_offsets = (int32_t *)mem(3), s.d_tiles = (int32_t *)mem(4);
                        s.d_order = (int32_t *)mem(5), s.d_place = (int32_t *)mem(6), s.d_ws = mem(7);
                        const size_t w = ecf_token_sort_workspace_bytes(E, k, T);
                        s.ws_bytes = w == SIZE_MAX ? 0 : w;
                        fine += ecf_token_sort(&s, T) == ECF_OK;
                        ecf_token_args t;
                        std::memset(&t, 0, sizeof t);
                        t.hidden = d, t.n_experts = E, t.top_k = k, t.dtype = dt, t.token_dtype = dt;
                        t.d_offsets = (int32_t *)mem(1), t.d_place = (int32_t *)mem(2), t.d_weight = (float *)mem(3);
                        t.d_x = mem(4), t.d_rows = mem(5), t.d_out = mem(6), t.d_dout = mem(7), t.d_drows = mem(8);
                        t.d_dweight = (float *)mem(9);
                        fine += ecf_token_dispatch(&t, T) == ECF_OK;
                        fine += ecf_token_combine(&t, T) == ECF_OK;
                        fine += ecf_token_combine_backward(&t, T) == ECF_OK;
                        ++done;
                    }
                for (int N : sizes)
                    for (int r : {1, 16, 64, 100, 256, 257}) {
                        ecf_adapter_args a;
                        std::memset(&a, 0, sizeof a);
                        a.in_features = d, a.out_features = N, a.rank = r, a.n_adapters = experts[done % 6];
                        a.dtype = a.wgrad_dtype = dt, a.out_dtype = done % 2 ? ECF_F32 : dt, a.idx_bytes = 4;
                        a.d_a = mem(1), a.d_b = mem(2), a.d_idx = mem(3), a.d_x = mem(4), a.d_h = (float *)mem(5);
                        a.d_out = mem(6), a.d_dout = mem(7), a.d_dx = mem(8), a.d_da = mem(9), a.d_db = mem(10), a.d_ws = mem(11);
                        for (int back = 0; back < 2; ++back) {
                            const size_t w = ecf_adapter_workspace_bytes(d, N, r, a.n_adapters, T, back);
                            a.ws_bytes = w == SIZE_MAX ? 0 : w;
                            fine += (back ? ecf_adapter_backward(&a, T) : ecf_adapter_forward(&a, T)) == ECF_OK;
                        }
                        ++done;
                    }
                token_host_launches();
            }
    std::printf("token checks passed: %ld shapes, %ld calls accepted\n", done, fine);
    return fine > 0 ? 0 : 1;
}
