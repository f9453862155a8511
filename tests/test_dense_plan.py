"""CPU tests of the dense operators' plan: which kernel each call takes, on 256 CUs.
The GPU tests pick their sizes so that between them every kernel runs; here the same
sizes go through the same plan, so that a change of its costs cannot leave a kernel
untested without a test failing."""
import math
import os
import random
import shutil
import subprocess

import pytest

import dense_host
import expert_cache_ffn_amd as ecf
import test_gpu_dense as G
import test_gpu_dense_kernels as GK


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    return dense_host.build(tmp_path_factory.mktemp("dense_host"))


def parameters(test, names):
    """The values a GPU test is parametrised with."""
    return next(m.args[1] for m in test.pytestmark if m.name == "parametrize" and m.args[0] == names)


def ok(r):
    assert r[0] == ecf.ECF_OK
    return [q for q in r[1] if q["kind"] != "grad"]


def layout(q):
    return "gated" if q["gated"] else "tn" if q["at"] else "nn" if q["bt"] else "nt"


def launched(host, dt):
    """Every product that the GPU tests of tiles, streaming, single gradients, short rows and the SIZES and LARGE
    lists run in type dt."""
    seen = []
    none = ecf.ECF_ACT_NONE
    if dt != "f32":
        for M, N, K in G.TILES:
            seen += ok(host.call("linear_forward", M, K, N, dt, none)) + ok(host.call("gated_forward", M, K, N, dt, none))
            seen += ok(host.call("linear_backward", M, N, K, dt, none, dw=False))
            seen += ok(host.call("linear_backward", K, N, M, dt, none, dx=False, db=False))
    for T, K, N in parameters(G.test_few_tokens, "T,K,N"):
        seen += ok(host.call("linear_forward", T, K, N, dt, out_dt="f32")) + ok(host.call("gated_forward", T, K, N, dt))
    for T, K, N in G.ONE:
        seen += ok(host.call("linear_backward", T, K, N, dt, none, dw=False))
        seen += ok(host.call("linear_backward", T, K, N, dt, none, dx=False)) + ok(host.call("linear_forward", T, K, N, dt, none))
        if N * K * T < 1 << 34:
            seen += ok(host.call("gated_forward", T, K, N, dt)) + ok(host.call("gated_backward", T, K, N, dt, dw=False))
            seen += ok(host.call("gated_backward", T, K, N, dt, dx=False, db=False))
    for T, K, N in GK.SPLIT_DW:
        seen += ok(host.call("linear_backward", T, K, N, dt, dx=False, gd="f32"))
    for T, d, n in G.SIZES + G.LARGE + parameters(G.test_gated_short_rows, "T,d,I"):
        for op in ("gated_forward", "gated_backward", "linear_forward", "linear_backward"):
            seen += ok(host.call(op, T, d, n, dt))
    return seen


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_the_gpu_tests_run_every_kernel(host, dt):
    seen = launched(host, dt)
    tiles = {(layout(q), q["dma"], q["tile"]) for q in seen if q["kind"] == "tiles"}
    kinds = [(0, 3)] if dt == "f32" else [(0, 4), (1, 5)]
    assert tiles == {(lay, dma, t) for lay in ("gated", "nt", "nn", "tn") for dma, n in kinds for t in range(n)}
    # both with and without a join, in every layout
    assert {(layout(q), q["splits"] > 1) for q in seen if q["kind"] == "tiles"} == {
        (lay, s) for lay in ("gated", "nt", "nn", "tn") for s in (False, True)}
    pairs = {(q["dma"], q["tile"]) for q in seen if q["kind"] == "pair"}
    assert pairs == ({(0, t) for t in range(3)} if dt == "f32" else {(0, 2), (0, 3), (1, 2), (1, 3), (1, 4)})
    few = {(q["gated"], q["rows"], q["groups"]) for q in seen if q["kind"] == "few"}
    assert few == {(g, r, t) for g in (0, 1) for r in (4, 8, 16) for t in (1, 2, 4)}
    assert {q["waves"] for q in seen if q["kind"] == "few"} == {1, 4, 8}
    assert {layout(q) for q in seen if q["kind"] == "short"} == {"gated", "nt", "nn", "tn"}


OPS = ("gated_forward", "gated_backward", "linear_forward", "linear_backward")


def drawn(n, seed):
    """Sizes over the whole range, their logarithms spread evenly, a multiple of 64 half of the time."""
    r = random.Random(seed)

    def size(hi):
        v = int(round(math.exp(r.uniform(0, math.log(hi)))))
        return v if r.random() < 0.5 else max(64, v // 64 * 64)

    for _ in range(n):
        yield r.choice(OPS), size(8192), size(16384), size(16384), r.choice(["f32", "bf16", "f16"])


def test_partial_sums_stay_in_their_workspace(host):
    """What a plan splits fits what the call was given, at the size the query names and not a byte less."""
    split = 0
    for op, T, d, n, dt in drawn(4000, 1):
        code, launches, need = host.call(op, T, d, n, dt)
        assert code == ecf.ECF_OK
        base = 62 * dense_host.APART
        for q in launches:
            if q["kind"] == "grad" or not q["room"]:
                assert q["kind"] == "grad" or not q.get("partials")
                continue
            assert base <= q["ws"] and q["ws"] + q["room"] <= base + need and q["ws"] % 256 == 0
            assert q.get("partials", 0) <= q["room"]
            if q["kind"] == "pair":
                assert q["at_w"] >= q["partials"] and q["at_w"] % 256 == 0
                assert not q["partials_w"] or q["at_w"] + q["partials_w"] <= q["room"]
            split += bool(q.get("partials"))
    assert split > 300


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("where", [dict(pad=1), dict(shift=1)])
def test_few_tokens_of_rows_at_odd_elements(host, where, dt):
    """16-bit rows that start at odd elements are read at less than half the rate by the streaming kernel: wide
    layers of up to 16 tokens go through tiles, though they have no workspace to split K in."""
    def kind(op, *size):
        launch, = ok(host.call(op, *size, dt, **where))
        assert launch["room"] == 0 and launch.get("splits", 1) == 1
        return launch["kind"]

    wide = "few" if dt == "f32" else "tiles"
    for op, *size in GK.ODD_ROWS:
        assert kind(op, *size) == wide
    for T, d, n in ((1, 4096, 1024), (16, 4096, 1024), (2, 128, 256), (16, 256, 64), (9, 640, 1500)):
        assert kind("linear_forward", T, d, n) == kind("gated_forward", T, d, n) == "few"
    # whole rows at even elements, whatever the size
    for op, *size in GK.ODD_ROWS:
        assert [q["kind"] for q in ok(host.call(op, *size, dt))] == ["few"]


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_host_code_under_sanitizers(tmp_path):
    exe = str(tmp_path / "dense_checks")
    subprocess.run(["g++", *dense_host.FLAGS, "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
                    *dense_host.SOURCES, os.path.join(dense_host.HERE, "sanitize", "dense_checks.cpp"), "-o", exe], check=True)
    p = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=600)
    assert p.returncode == 0 and "dense checks passed" in p.stdout, p.stdout[-4000:]
    for bad in ("ERROR: AddressSanitizer", "runtime error:"):
        assert bad not in p.stdout, p.stdout[-4000:]


def test_small_layers_ask_for_small_workspaces(host):
    """No more than dz, the bias sums and what the products of these sizes can split into."""
    for dt in ("f32", "bf16", "f16"):
        for op in ("gated_backward", "linear_backward"):
            assert host.call(op, 64, 256, 128, dt)[2] < 1 << 20
            assert host.call(op, 8, 64, 64, dt)[2] < 1 << 16
            # reductions under two k-tiles of 64 are not split
            assert host.call(op, 100, 4096, 60, dt)[2] < 100 * 64 * 2 * 4 + 8 * 64 * 2 * 4 + 8192 + 2 * 4 * 100 * 4096 * 4
    assert host.call("linear_forward", 500, 100, 5000, "bf16")[2] == 0
    big = host.call("linear_backward", 8192, 2048, 4096, "bf16")[2]
    assert 8192 * 4096 * 2 < big <= 8192 * 4096 * 2 + 256 * 4096 * 4 + (32 << 20) + 4096


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_no_workspace_for_a_dz_that_is_dy(host, dt):
    """Without an activation and in the operands' type, nothing is written for dz and nothing asked for it."""
    none, T, K, N = ecf.ECF_ACT_NONE, 8192, 2048, 4096
    code, launches, need = host.call("linear_backward", T, K, N, dt, none, want_ws=2)
    assert code == ecf.ECF_OK and need <= (T // 32) * N * 4 + (32 << 20) + 8192
    assert all(q["dz"] == 0 if q["kind"] == "grad" else q["a0"] == 4 * dense_host.APART for q in launches)  # dout's place
    assert host.call("linear_backward", T, K, N, dt, none, want_ws=2, ws=need - 1)[0] == ecf.ECF_ENOSPC
    # the larger size serves it too, and is what every other call needs
    full = host.call("linear_backward", T, K, N, dt, none)[2]
    assert full >= need + T * N * dense_host.SIZE[dt]
    assert host.call("linear_backward", T, K, N, dt, none)[0] == ecf.ECF_OK
    assert host.call("linear_backward", T, K, N, dt, ecf.ECF_ACT_RELU, ws=need)[0] == ecf.ECF_ENOSPC
    if dt != "f32":
        assert host.call("linear_backward", T, K, N, dt, none, out_dt="f32", ws=need)[0] == ecf.ECF_ENOSPC


def test_backward_buffers_lie_apart(host):
    """Column sums, what the scales are found from and their inverses, partial sums and dz, in the workspace and not
    on one another."""
    base = 62 * dense_host.APART
    for op, T, d, n, dt in drawn(2000, 5):
        if not op.endswith("backward"):
            continue
        # (a linear dz of an fp16 dy is dy, or through relu dy and zeros)
        scaled = (ecf.ECF_ACT_SILU, ecf.ECF_ACT_NONE, ecf.ECF_ACT_RELU)[: 3 if op[0] == "g" else 1]
        for act in (ecf.ECF_ACT_SILU, ecf.ECF_ACT_NONE, ecf.ECF_ACT_RELU):
            code, launches, need = host.call(op, T, d, n, dt, act)
            assert code == ecf.ECF_OK
            halves, e, pitch = 1 + (op[0] == "g"), dense_host.SIZE[dt], (n + 7) // 8 * 8
            spans = []
            for q in launches:
                if q["kind"] == "grad":
                    spans.append((q["partial"], (T + 31) // 32 * halves * n * 4))
                    spans += [(q[z], T * pitch * halves * e) for z in ("dz", "dz_w") if q[z]]
                    assert q["scaled"] == (dt == "f16" and act in scaled) and bool(q["dz_w"]) == q["scaled"]
                    if q["scaled"]:
                        spans += [(q["row_tops"], (n + 63) // 64 * T * 4), (q["col_tops"], (T + 31) // 32 * halves * n * 4),
                                  (q["row_inverse"], T * 4), (q["col_inverse"], halves * n * 4)]
                else:
                    assert bool(q["unscale"]) == (dt == "f16" and act in scaled)
                if q.get("partials") or q.get("partials_w"):
                    spans.append((q["ws"], q["room"]))
            spans = sorted(set(spans))
            assert all(at >= base and at % 256 == 0 and at + size <= base + need for at, size in spans)
            assert all(p[0] + p[1] <= q[0] for p, q in zip(spans, spans[1:]))


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_no_tokens_read_no_scale(host, dt):
    """Without tokens no scale is written, so none may be read: zeros times what the workspace held are not zeros."""
    for op in ("gated_backward", "linear_backward"):
        code, launches, _ = host.call(op, 0, 64, 40, dt, gd="f32")
        assert code == ecf.ECF_OK
        products = [q for q in launches if q["kind"] != "grad"]
        assert products and all(q["unscale"] == 0 for q in products)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_wide_layers_are_refused_by_the_stated_limit_alone(host, dt):
    """256 rows of every operand under 2 GiB: what meets that runs, and the size query refuses the widths whose
    rows alone do not."""
    limit = ((1 << 31) - 1) // 256 // dense_host.SIZE[dt]  # elements
    for op in OPS:
        for d, n in ((8, 1 << 20), (8, limit), (8, limit - 6), (limit, 8), (1 << 20, 1 << 20), (limit, limit)):
            code, _, need = host.call(op, 5, d, n, dt)
            assert code == ecf.ECF_OK and need < 1 << 62, (op, d, n, host.error())
        for d, n in ((8, limit + 1), (limit + 1, 8)):
            code, _, need = host.call(op, 5, d, n, dt)
            assert code != ecf.ECF_OK and need == (1 << 64) - 1, (op, d, n)
