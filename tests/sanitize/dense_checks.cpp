// A sweep of the dense operators' entry points and plan under the sanitizers: sizes
// from one to the largest, every type, odd strides, missing operands, on stub launchers.
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "../../include/ecf.h"

extern "C" const char *dense_host_launches();
extern "C" void dense_host_cus(int cus);

int main()
{
    const int sizes[] = {1, 2, 7, 8, 31, 63, 64, 65, 130, 1000, 4096, 16384, 200001, 1 << 21, 1 << 22, 0, -1, (1 << 22) + 1};
    const int tokens[] = {0, 1, 3, 16, 17, 64, 65, 500, 8192, 1 << 22, -1};
    long done = 0, fine = 0;
    char *base = (char *)((size_t)1 << 40);
    for (int cus : {256, 1, 304})
        for (int dt : {ECF_F32, ECF_BF16, ECF_F16, ECF_MXFP4})
            for (int d : sizes)
                for (int n : sizes)
                    for (int T : tokens) {
                        dense_host_cus(cus);
                        ecf_gated_args g;
                        ecf_linear_args l;
                        std::memset(&g, 0, sizeof g);
                        std::memset(&l, 0, sizeof l);
                        const size_t step = (size_t)1 << 36;
                        g.hidden = l.in_features = d, g.inter = l.out_features = n;
                        g.dtype = l.dtype = l.out_dtype = g.wgrad_dtype = l.wgrad_dtype = dt;
                        g.act = l.act = (int)(done % 5);
                        g.d_x = l.d_x = base, g.d_w_gate = l.d_w = base + step, g.d_w_up = base + 2 * step;
                        g.d_h = l.d_out = base + 3 * step;
                        g.ld_x = l.ld_x = done % 3 ? 0 : d + 1;
                        for (int back = 0; back < 2; ++back) {
                            const size_t wg = ecf_gated_workspace_bytes(d, n, dt, T, back);
                            const size_t wl = ecf_linear_workspace_bytes(d, n, dt, T, back);
                            g.d_ws = l.d_ws = base + 4 * step;
                            g.ws_bytes = wg == SIZE_MAX ? 0 : wg, l.ws_bytes = wl == SIZE_MAX ? 0 : wl;
                            if (!back) {
                                fine += ecf_gated_forward(&g, T) == ECF_OK;
                                fine += ecf_linear_forward(&l, T) == ECF_OK;
                                continue;
                            }
                            g.d_a = l.d_z = base + 5 * step, g.d_b = base + 6 * step, g.d_dh = l.d_dout = base + 7 * step;
                            g.d_dx = l.d_dx = base + 8 * step;
                            g.d_dw_gate = l.d_dw = base + 9 * step, g.d_dw_up = base + 10 * step;
                            fine += ecf_gated_backward(&g, T) == ECF_OK;
                            fine += ecf_linear_backward(&l, T) == ECF_OK;
                        }
                        dense_host_launches();
                        ++done;
                    }
    std::printf("dense checks passed: %ld shapes, %ld calls accepted\n", done, fine);
    return fine > 0 ? 0 : 1;
}
