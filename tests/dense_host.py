"""The dense operators' host code on the CPU: dense.cpp and dense_plan.cpp built with
g++ around stub launchers (sanitize/dense_host.cpp), called with addresses that
nothing dereferences.  A call returns its code and what it would have launched."""
import ctypes
import json
import os
import subprocess

import expert_cache_ffn_amd as ecf

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "expert_cache_ffn_amd", "csrc")
SOURCES = [os.path.join(CSRC, "dense.cpp"), os.path.join(CSRC, "dense_plan.cpp"), os.path.join(HERE, "sanitize", "dense_host.cpp")]
FLAGS = ["-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include"]
DT = {"f32": ecf.ECF_F32, "bf16": ecf.ECF_BF16, "f16": ecf.ECF_F16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
APART = 1 << 38  # between the made-up operands


def build(folder):
    out = os.path.join(str(folder), "libdense_host.so")
    subprocess.run(["g++", *FLAGS, "-fPIC", "-shared", *SOURCES, "-o", out], check=True)
    return Host(out)


class Host:
    def __init__(self, path):
        L = self.lib = ctypes.CDLL(path)
        L.dense_host_launches.restype = L.dense_host_error.restype = ctypes.c_char_p
        for name, args in (("gated", ecf.GatedArgs), ("linear", ecf.LinearArgs)):
            ws = getattr(L, f"ecf_{name}_workspace_bytes")
            ws.argtypes, ws.restype = [ctypes.c_int32] * 5, ctypes.c_size_t
            for way in ("forward", "backward"):
                getattr(L, f"ecf_{name}_{way}").argtypes = [ctypes.POINTER(args), ctypes.c_int32]

    def error(self):
        return self.lib.dense_host_error().decode()

    def call(self, op, T, d, n, dt, act=ecf.ECF_ACT_SILU, out_dt=None, dx=True, dw=True, db=True, shift=0, pad=0, ws=None,
             gd=None, want_ws=None):
        """(code, launches, workspace bytes): op "gated_forward" and so on, rows `pad` elements further apart than
        they are long, starting `shift` elements into their memory; ws: workspace bytes, want_ws: the size query's
        last argument."""
        name, way = op.split("_")
        back = way == "backward"
        e, dtype = SIZE[dt], DT[dt]
        need = getattr(self.lib, f"ecf_{name}_workspace_bytes")(d, n, dtype, T, int(back) if want_ws is None else want_ws)
        a = ecf.GatedArgs() if name == "gated" else ecf.LinearArgs()
        at = iter(range(1, 64))

        def mem():
            return next(at) * APART + shift * e

        a.dtype, a.act, a.wgrad_dtype = dtype, act, dtype if gd is None else DT[gd]
        if name == "gated":
            a.hidden, a.inter = d, n
            a.d_x, a.d_w_gate, a.d_w_up, a.d_a, a.d_b, a.d_dh = (mem() for _ in range(6))
            a.ld_x = a.ld_w = d + pad
            a.ld_ab = a.ld_dh = n + pad
            if not back:
                a.d_h, a.d_a, a.d_b = mem(), None, None
        else:
            a.in_features, a.out_features = d, n
            a.out_dtype = dtype if out_dt is None else DT[out_dt]
            a.d_x, a.d_w, a.d_z, a.d_dout = (mem() for _ in range(4))
            a.ld_x = a.ld_w = d + pad
            a.ld_z = a.ld_dout = n + pad
            if not back:
                a.d_out, a.d_z = mem(), None
        if back:
            wide = next(at) * APART  # (gradients of either type)
            if dx:
                a.d_dx = mem()
            if dw and name == "gated":
                a.d_dw_gate, a.d_dw_up = wide, wide + APART // 2
                if db:
                    a.d_db_gate, a.d_db_up = wide + APART // 4, wide + APART // 4 * 3
            elif dw:
                a.d_dw = wide
                if db:
                    a.d_dbias = wide + APART // 2
        have = need if ws is None else ws
        if have and have != ctypes.c_size_t(-1).value:
            a.d_ws, a.ws_bytes = 62 * APART, have
        code = getattr(self.lib, "ecf_" + op)(ctypes.byref(a), T)
        return code, json.loads(self.lib.dense_host_launches()), need
