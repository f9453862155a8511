"""The token operators' host code on the CPU: tokens.cpp and adapters.cpp built with g++ around stub launchers
(sanitize/tokens_host.cpp), called with addresses that nothing dereferences."""
import ctypes
import json
import os
import subprocess

import expert_cache_ffn_amd as ecf

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "expert_cache_ffn_amd", "csrc")
SOURCES = [os.path.join(CSRC, "tokens.cpp"), os.path.join(CSRC, "adapters.cpp"), os.path.join(HERE, "sanitize", "tokens_host.cpp")]
FLAGS = ["-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include"]
APART = 1 << 40  # between the made-up operands
WS = 60 * APART


def build(folder):
    out = os.path.join(str(folder), "libtokens_host.so")
    subprocess.run(["g++", *FLAGS, "-fPIC", "-shared", *SOURCES, "-o", out], check=True)
    return Host(out)


class Host:
    def __init__(self, path):
        L = self.lib = ctypes.CDLL(path)
        L.token_host_launches.restype = L.token_host_error.restype = ctypes.c_char_p
        for name, n in (("norm", 3), ("token_sort", 3), ("adapter", 6)):
            f = getattr(L, f"ecf_{name}_workspace_bytes")
            f.argtypes, f.restype = [ctypes.c_int32] * n, ctypes.c_size_t

    def run(self, name, args, T):
        """What the call would have launched."""
        code = getattr(self.lib, name)(ctypes.byref(args), T)
        assert code == ecf.ECF_OK, self.lib.token_host_error().decode()
        return json.loads(self.lib.token_host_launches())

    def grid(self, blocks):
        x, y = ctypes.c_uint32(), ctypes.c_uint32()
        self.lib.token_host_grid(ctypes.c_int64(blocks), ctypes.byref(x), ctypes.byref(y))
        return x.value, y.value

    def norm_backward(self, T, d, ws=None):
        a = ecf.NormArgs()
        a.hidden = d
        for i, f in enumerate(("d_sum", "d_rstd", "d_dy", "d_dx", "d_dweight")):
            setattr(a, f, (i + 1) * APART)
        a.d_ws, a.ws_bytes = WS, ws or self.lib.ecf_norm_workspace_bytes(d, T, 1)
        return self.run("ecf_norm_backward", a, T), a.ws_bytes

    def sort(self, T, k, E, ws=None):
        a = ecf.SortArgs()
        a.n_experts, a.top_k, a.idx_bytes = E, k, 4
        for i, f in enumerate(("d_idx", "d_counts", "d_offsets", "d_tiles", "d_order", "d_place")):
            setattr(a, f, (i + 1) * APART)
        a.d_ws, a.ws_bytes = WS, ws or self.lib.ecf_token_sort_workspace_bytes(E, k, T)
        return self.run("ecf_token_sort", a, T), a.ws_bytes

    def adapters(self, T, K, N, r, n, back, order=False, out_dtype=ecf.ECF_BF16, ws=None):
        a = ecf.AdapterArgs()
        a.in_features, a.out_features, a.rank, a.n_adapters, a.idx_bytes = K, N, r, n, 4
        a.dtype = a.wgrad_dtype = ecf.ECF_BF16
        a.out_dtype = out_dtype
        names = ["d_a", "d_b", "d_idx", "d_x", "d_h"] + (["d_dout", "d_dx", "d_da", "d_db"] if back else ["d_out"])
        for i, f in enumerate(names + (["d_order", "d_offsets", "d_tiles"] if order else [])):
            setattr(a, f, (i + 1) * APART)
        a.d_ws, a.ws_bytes = WS, ws or self.lib.ecf_adapter_workspace_bytes(K, N, r, n, T, int(back))
        return self.run(f"ecf_adapter_{'backward' if back else 'forward'}", a, T), a.ws_bytes


def overlaps(parts, end):
    """Whether one of the parts [(name, address, bytes)] of a workspace of `end` bytes leaves it or meets another: their names."""
    parts = sorted((p for p in parts if p[2]), key=lambda p: p[1])
    bad = [p for p in parts if p[1] < WS or p[1] + p[2] > WS + end]
    return bad + [(p, q) for p, q in zip(parts, parts[1:]) if p[1] + p[2] > q[1]]
